"""Where the binding's allocations belong when a call is given a stream (no GPU: the library is replaced by one that
answers BQ_OK, and torch.cuda.stream by one that remembers)."""
import contextlib

import pytest
import torch

import bit_quantized_linear_rmsnorm_b200 as bq


class Stream:
    cuda_stream = 0


class Library:
    """Every call succeeds; every size is 64 bytes."""

    def __getattr__(self, name):
        return lambda *args: 64 if "bytes" in name else bq.BQ_OK


def f(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


i8, i32, u8, f32 = torch.int8, torch.int32, torch.uint8, torch.float32
CALLS = {
    "bq_act_quant_int8": (3, lambda **kw: bq.bq_act_quant_int8(f(4, 64), **kw)),
    "bq_act_quant_int8_layernorm": (3, lambda **kw: bq.bq_act_quant_int8_layernorm(f(4, 64), **kw)),
    "bq_bitlinear_w2a8_layernorm": (2, lambda **kw: bq.bq_bitlinear_w2a8_layernorm(
        f(4, 64), f(8, 4, dtype=i32), f(1, dtype=f32), 8, **kw)),
    "bq_weight_quant_ternary_pack": (3, lambda **kw: bq.bq_weight_quant_ternary_pack(f(8, 64), **kw)),
    "bq_weight_pack_int4_grouped": (2, lambda **kw: bq.bq_weight_pack_int4_grouped(
        f(8, 128, dtype=u8), f(8, 1, dtype=u8), 128, **kw)),
    "bq_gemm_i8_pertoken": (1, lambda **kw: bq.bq_gemm_i8_pertoken(
        f(4, 64, dtype=i8), f(8, 64, dtype=i8), f(8, dtype=f32), f(4, dtype=f32), **kw)),
    "bq_gemm_i8_pertoken_batched": (1, lambda **kw: bq.bq_gemm_i8_pertoken_batched(
        f(2, 4, 64, dtype=i8), f(2, 8, 64, dtype=i8), f(8, dtype=f32), f(4, dtype=f32), **kw)),
    "bq_bitlinear_w2a8": (2, lambda **kw: bq.bq_bitlinear_w2a8(
        f(4, 64), f(8, 4, dtype=i32), f(1, dtype=f32), 8, **kw)),
    "bq_bitlinear_w2a8_noalloc": (1, lambda **kw: bq.bq_bitlinear_w2a8_noalloc(
        f(4, 64), f(8, 4, dtype=i32), f(1, dtype=f32), 8, **kw)),
    "bq_linear_w4_grouped": (2, lambda **kw: bq.bq_linear_w4_grouped(
        f(4, 128, dtype=f32), f(8, 16, dtype=i32), f(8, 1, dtype=torch.int16), f(8, 1, dtype=i32), 128, **kw)),
    "bq_weight_quant_int4_pack": (1, lambda **kw: bq.bq_weight_quant_int4_pack(f(8, 64), f(1, dtype=f32), 1e-5, **kw)),
    "bq_act_quant_int4": (1, lambda **kw: bq.bq_act_quant_int4(f(4, 64), f(1, dtype=f32), 1e-5, **kw)),
    "bq_linear_w4a4": (2, lambda **kw: bq.bq_linear_w4a4(
        f(4, 64), f(1, dtype=f32), f(8, 8, dtype=i32), f(1, dtype=f32), 8, 1e-5, **kw)),
    "bq_bitconv1d_weight_pack": (3, lambda **kw: bq.bq_bitconv1d_weight_pack(f(8, 64, 3), **kw)),
    "bq_bitconv1d": (2, lambda **kw: bq.bq_bitconv1d(
        f(2, 64, 32), f(3, 8, 4, dtype=i32), f(1, dtype=f32), 8, 3, **kw)),
    "bq_bitlinear_w2a8_backward": (3, lambda **kw: bq.bq_bitlinear_w2a8_backward(
        f(4, 64), f(4, 8), f(8, 4, dtype=i32), f(1, dtype=f32), **kw)),
    "bq_linear_w4a4_backward": (4, lambda **kw: bq.bq_linear_w4a4_backward(
        f(4, 64), f(8, 64), f(4, 8), f(1, dtype=f32), f(1, dtype=f32), 1e-5, **kw)),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_follow_the_stream(monkeypatch, name):
    """Outputs and workspaces that a call makes belong to the stream that it launches on: on the current stream the
    allocator could hand them out again while the call's kernels still use them."""
    count, call = CALLS[name]
    mine, inside, made = Stream(), [], []
    empty = torch.empty

    @contextlib.contextmanager
    def enter(stream):
        inside.append(stream)
        yield
        inside.pop()

    def watched(*args, **kw):
        made.append(inside[-1] if inside else None)
        return empty(*args, **kw)

    monkeypatch.setattr(bq, "lib", Library)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch, "empty", watched)
    call(stream=mine)
    assert made == [mine] * count


def test_a_copy_follows_the_stream(monkeypatch):
    """A weight that has to be made dense first is copied on the call's stream as well."""
    seen = []

    @contextlib.contextmanager
    def enter(stream):
        seen.append(stream)
        yield

    mine = Stream()
    monkeypatch.setattr(bq, "lib", Library)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    w = f(3, 64, 8).permute(2, 1, 0)
    bq.bq_bitconv1d_weight_pack(w, wpacked=f(3, 8, 4, dtype=i32), w_scale=f(1, dtype=f32),
                                workspace=f(64, dtype=u8), stream=mine)
    assert seen == [mine]
