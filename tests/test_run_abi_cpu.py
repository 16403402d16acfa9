"""The calls of gptq_run.h: exported, bound, and refusing bad arguments on the
host (no GPU is touched: the addresses are never dereferenced)."""
import ctypes
import os
import re

import pytest

from post_weight_quantization_layer_amd import binding as B
from post_weight_quantization_layer_amd import binding_run as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000          # a plausible address, 256-byte aligned
BAD, WS, OK = B.GPTQ_ERR_INVALID_ARG, B.GPTQ_ERR_WORKSPACE, B.GPTQ_OK
F32, BF16, F16 = 0, 1, 2


def said(word):
    return word in B.gptq_last_error()


def test_every_declared_call_is_exported_and_bound():
    with open(os.path.join(ROOT, "include", "gptq_run.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(gptq_[a-z0-9_]+)\s*\(", text))
    assert names == set(R.EXPORTED)
    for n in names:
        assert getattr(R.lib(), n).argtypes is not None, n


def test_sizes():
    L = R.lib()
    assert [L.gptq_tokens_ld(c) for c in (0, 1, 128, 129, 65536, 65537, -5)] == \
        [0, 128, 128, 256, 65536, 0, 0]
    assert L.gptq_w8a8_layer_bytes(17, 129) >= 32 * 256 + 2 * 32 * 4
    assert L.gptq_w8a8_layer_bytes(1 << 19, 65536) > 1 << 35
    for bad in ((0, 5), (5, 0), (5, 65537), ((1 << 24) + 1, 5), ((1 << 19) + 1, 65536)):
        assert L.gptq_w8a8_layer_bytes(*bad) == 0
    assert L.gptq_w8a8_linear_ws_bytes(None, 4) == 0
    assert L.gptq_token_logprobs_ws_bytes(0, 100, 5) == 0
    assert L.gptq_token_logprobs_ws_bytes(10, 100, 65) == 0
    with pytest.raises(B.GptqError):
        R.gptq_tokens_ld(65537)


@pytest.mark.parametrize("change,word", [
    (dict(x=None), "x must not be NULL"), (dict(x=A + 1), "aligned"), (dict(dtype=7), "type"),
    (dict(tokens=-1), "tokens"), (dict(tokens=(1 << 21) + 1), "tokens"),
    (dict(cols=0), "cols"), (dict(cols=70000), "cols"),
    (dict(ld_x=299), "stride"), (dict(codes=None), "NULL"), (dict(codes=A + 8), "16-byte"),
    (dict(ld_codes=300), "ld_codes"), (dict(ld_codes=392), "ld_codes"), (dict(scale=None), "NULL"),
    (dict(sum=A + 2), "4-byte")])
def test_quantize_refuses(change, word):
    a = dict(x=A, dtype=F16, tokens=4, cols=300, ld_x=300, codes=A, ld_codes=384, scale=A, sum=A)
    a.update(change)
    st = R.lib().gptq_quantize_tokens(a["x"], a["dtype"], a["tokens"], a["cols"], a["ld_x"],
                                      a["codes"], a["ld_codes"], a["scale"], a["sum"], None)
    assert st == BAD and said(word), B.gptq_last_error()
    if "x" in change:
        for g, u in ((a["x"], A), (A, a["x"])):
            assert R.lib().gptq_silu_mul_quantize(g, u, F16, 4, 300, 300, A, 384, A, A, None) == BAD


def layer(rows=64, cols=300, mem=A, nbytes=None):
    n = R.lib().gptq_w8a8_layer_bytes(rows, cols)
    return R.gptq_w8a8_layer(rows, cols, (rows + 15) // 16 * 16, (cols + 127) // 128 * 128, mem,
                             n if nbytes is None else nbytes)


@pytest.mark.parametrize("change,word", [
    (dict(q=None), "NULL"), (dict(rows=0), "rows"), (dict(cols=65537), "cols"),
    (dict(mem=A + 64), "256-byte"), (dict(nbytes=100), "too small"), (dict(scale=A + 1), "aligned"),
    (dict(zero=None), "NULL")])
def test_prepare_refuses(change, word):
    a = dict(q=A, scale=A, zero=A, rows=64, cols=300, mem=A, nbytes=1 << 20)
    a.update(change)
    out = R.gptq_w8a8_layer()
    st = R.lib().gptq_w8a8_prepare(a["q"], a["scale"], a["zero"], a["rows"], a["cols"], a["mem"],
                                   a["nbytes"], out, None)
    assert st == BAD and said(word) and out.rows == 0


@pytest.mark.parametrize("change,status,word", [
    (dict(layer=None), BAD, "prepared"), (dict(layer=layer(mem=None)), BAD, "prepared"),
    (dict(layer=layer(nbytes=8)), BAD, "prepared"), (dict(x=None), BAD, "NULL"),
    (dict(dtype=9), BAD, "type"), (dict(ld_x=10), BAD, "stride"), (dict(tokens=-1), BAD, "tokens"),
    (dict(tokens=(1 << 20) + 1), BAD, "tokens"), (dict(y=None), BAD, "y must"),
    (dict(y_dtype=3), BAD, "type"), (dict(y=A + 1), BAD, "aligned"), (dict(ld_y=63), BAD, "ld_y"),
    (dict(ws=None), WS, "NULL"), (dict(ws=A + 16), WS, "256-byte"), (dict(n=64), WS, "too small")])
def test_linear_refuses(change, status, word):
    a = dict(layer=layer(), x=A, dtype=BF16, ld_x=300, tokens=4, y=A, y_dtype=F16, ld_y=64, ws=A,
             n=1 << 30)
    a.update(change)
    st = R.lib().gptq_w8a8_linear(a["layer"], a["x"], a["dtype"], a["ld_x"], a["tokens"], a["y"],
                                  a["y_dtype"], a["ld_y"], a["ws"], a["n"], None)
    assert st == status and said(word), B.gptq_last_error()


@pytest.mark.parametrize("change,word", [
    (dict(codes=None), "NULL"), (dict(codes=A + 4), "16-byte"), (dict(ld_codes=383), "ld_codes"),
    (dict(ld_codes=256), "ld_codes"), (dict(scale=None), "NULL"), (dict(sum=A + 1), "4-byte")])
def test_gemm_refuses(change, word):
    a = dict(codes=A, ld_codes=384, scale=A, sum=A)
    a.update(change)
    st = R.lib().gptq_w8a8_gemm(layer(), a["codes"], a["ld_codes"], a["scale"], a["sum"], 4, A, F16,
                                64, A, 1 << 30, None)
    assert st == BAD and said(word), B.gptq_last_error()


@pytest.mark.parametrize("change,word", [
    (dict(post=3), "post and pre"), (dict(pre=-1), "post and pre"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(w_dtype=5), "w_dtype"), (dict(post_weight=A + 1), "aligned"),
    (dict(d=0), "d must"), (dict(d=32769), "d must"), (dict(dtype=4), "type"), (dict(r=None), "r must"),
    (dict(ld_r=63), "stride"), (dict(ld_b=63), "stride"), (dict(b=A + 1), "aligned"),
    (dict(gate_tokens=0), "gate_tokens"), (dict(ld_gate=3), "stride"),
    (dict(r_out=None, h=None, codes=None), "one of"), (dict(ld_h=1), "stride"),
    (dict(codes=A + 1), "16-byte"), (dict(ld_codes=64), "ld_codes"), (dict(scale=None), "NULL")])
def test_norm_block_refuses(change, word):
    a = dict(post=1, pre=1, w_dtype=F16, eps=1e-6, post_weight=A, d=64, dtype=F16, r=A, ld_r=64,
             b=A, ld_b=64, gate=A, ld_gate=64, gate_tokens=1, r_out=A, h=A, ld_h=64, codes=A,
             ld_codes=128, scale=A, sum=A)
    a.update(change)
    p = R.gptq_norm_params(a["post"], a["pre"], a["w_dtype"], a["eps"], 0.0, 1.0, 1.0,
                           a["post_weight"], None, None, None)
    st = R.lib().gptq_norm_block(p, a["dtype"], 4, a["d"], a["r"], a["ld_r"], a["b"], a["ld_b"],
                                 a["gate"], a["ld_gate"], a["gate_tokens"], a["r_out"], 64, a["h"],
                                 a["ld_h"], a["codes"], a["ld_codes"], a["scale"], a["sum"], None)
    assert st == BAD and said(word), B.gptq_last_error()
    assert R.lib().gptq_norm_block(None, F16, 4, 64, A, 64, None, 0, None, 0, 1, A, 64, None, 0,
                                   None, 0, None, None, None) == BAD


@pytest.mark.parametrize("change,status,word", [
    (dict(logits=None), BAD, "logits"), (dict(logits=A + 1), BAD, "aligned"),
    (dict(ids=A + 4), BAD, "aligned"), (dict(dtype=8), BAD, "type"), (dict(rows=-1), BAD, "rows"),
    (dict(rows=(1 << 23) + 1), BAD, "rows"),
    (dict(vocab=0), BAD, "vocab"), (dict(vocab=(1 << 24) + 1), BAD, "vocab"), (dict(ld=999), BAD, "ld"),
    (dict(scale=0.0), BAD, "scale"), (dict(scale=1e31), BAD, "scale"),
    (dict(scale=float("inf")), BAD, "scale"),
    (dict(scale=float("nan")), BAD, "scale"), (dict(k=65), BAD, "top_k"),
    (dict(k=20, vocab=10, ld=10), BAD, "top_k"), (dict(top_ids=None), BAD, "top_ids"),
    (dict(ids=None), BAD, "ids"), (dict(entropy=A + 2), BAD, "aligned"),
    (dict(ws=None, vocab=100000, ld=100000), WS, "NULL"),
    (dict(ws=A + 8, vocab=100000, ld=100000), WS, "256-byte"),
    (dict(n=16, vocab=100000, ld=100000), WS, "too small")])
def test_token_logprobs_refuses(change, status, word):
    a = dict(logits=A, dtype=F32, rows=4, vocab=1000, ld=1000, ids=A, scale=1.0, k=5, entropy=A,
             top_ids=A, ws=A, n=1 << 30)
    a.update(change)
    st = R.lib().gptq_token_logprobs(a["logits"], a["dtype"], a["rows"], a["vocab"], a["ld"],
                                     a["ids"], a["scale"], a["k"], A, A, a["entropy"], a["top_ids"],
                                     A, a["ws"], a["n"], None)
    assert st == status and said(word), B.gptq_last_error()


def gated_mlp(enter=None, up=None, down=None):
    norm = R.gptq_norm_params(0, 1, F16, 1e-6, 0.0, 1.0, 1.0, None, None, None, None)
    return R.gptq_gated_mlp(enter or norm, norm, up or layer(600, 64), down or layer(64, 300))


@pytest.mark.parametrize("change,status,word", [
    (dict(mlp=None), BAD, "prepared"), (dict(mlp=gated_mlp(up=layer(600, 65))), BAD, "down.rows"),
    (dict(mlp=gated_mlp(down=layer(64, 301))), BAD, "2 down.cols"),
    (dict(mlp=gated_mlp(up=layer(600, 64, mem=None))), BAD, "prepared"),
    (dict(dtype=4), BAD, "dtype"), (dict(tokens=-1), BAD, "tokens"),
    (dict(tokens=(1 << 20) + 1), BAD, "tokens"), (dict(r_out=None, h=None), BAD, "one of"),
    (dict(ws=None), WS, "NULL"), (dict(ws=A + 16), WS, "256-byte"), (dict(n=4096), WS, "too small"),
    (dict(r=None), BAD, "r must"), (dict(ld_r=63), BAD, "stride"),
    (dict(mlp=gated_mlp(enter=R.gptq_norm_params(0, 7, F16, 1e-6, 0.0, 1.0, 1.0, None, None, None,
                                                 None))), BAD, "post and pre")])
def test_gated_mlp_refuses(change, status, word):
    a = dict(mlp=gated_mlp(), dtype=F16, tokens=4, r=A, ld_r=64, r_out=A, h=A, ws=A, n=1 << 30)
    a.update(change)
    st = R.lib().gptq_gated_mlp_forward(a["mlp"], a["dtype"], a["tokens"], a["r"], a["ld_r"], None,
                                        0, 1, a["r_out"], 64, a["h"], 64, a["ws"], a["n"], None)
    assert st == status and said(word), B.gptq_last_error()


def test_gated_mlp_scratch():
    f = R.lib().gptq_gated_mlp_ws_bytes
    # codes of 4 rows of 128 and 384, 4 x 600 and 4 x 64 values
    assert f(gated_mlp(), F16, 4) >= 4 * (128 + 384) + 2 * 4 * 664
    assert f(gated_mlp(), F32, 4) > f(gated_mlp(), F16, 4)
    assert f(None, F16, 4) == f(gated_mlp(), 9, 4) == f(gated_mlp(), F16, 0) == 0


def test_zero_tokens_are_no_ops():
    L = R.lib()
    p = R.gptq_norm_params(1, 1, F16, 1e-6, 0.0, 1.0, 1.0, None, None, None, None)
    assert L.gptq_quantize_tokens(None, F16, 0, 300, 300, None, 0, None, None, None) == OK
    assert L.gptq_silu_mul_quantize(None, None, F16, 0, 300, 300, None, 0, None, None, None) == OK
    assert L.gptq_w8a8_linear(layer(), None, F16, 300, 0, None, F16, 64, None, 0, None) == OK
    assert L.gptq_w8a8_gemm(layer(), None, 0, None, None, 0, None, F16, 64, None, 0, None) == OK
    assert L.gptq_norm_block(p, F16, 0, 64, None, 64, None, 0, None, 0, 1, None, 64, None, 0, None,
                             0, None, None, None) == OK
    assert L.gptq_gated_mlp_forward(gated_mlp(), F16, 0, None, 64, None, 0, 1, None, 64, None, 64,
                                    None, 0, None) == OK
    assert L.gptq_token_logprobs(None, F32, 0, 100, 100, None, 1.0, 0, None, None, None, None,
                                 None, None, 0, None) == OK


def test_classes_refuse():
    torch = pytest.importorskip("torch")
    from post_weight_quantization_layer_amd.norms import NormBlock
    from post_weight_quantization_layer_amd.scoring import TokenScorer
    from post_weight_quantization_layer_amd.w8a8 import W8A8Linear, quantize_tokens
    cpu = torch.zeros((4, 8))
    for call in (lambda: quantize_tokens(cpu), lambda: NormBlock(8)(cpu),
                 lambda: NormBlock(8, pre="rms", pre_weight=torch.zeros(8)),
                 lambda: TokenScorer(4, 8, 9, device="cpu"), lambda: TokenScorer(4, 8, 2, device="cpu")(cpu),
                 lambda: W8A8Linear(cpu, cpu, cpu), lambda: quantize_tokens(cpu.t())):
        with pytest.raises(ValueError):
            call()
