"""Refusals of the block-scaled calls that take lengths at a stride.  On the
host, before any CUDA call, so fake addresses are never dereferenced."""
import pytest
import torch

A = 0x10000          # 16-byte aligned


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import build
    build.build()
    from paged_kv_cache_455_b200 import pa as mod
    return mod


def _append(pa, stride, T=9, bs=16):
    return pa.lib.pa_rope_and_cache_q8_strided(A, 1024, A, 1024, A, 256, A, 256, A, A, A, A, A, T, 4,
                                               A, 4, A, stride, 3, A, A, 64, 100, 0, 8, 2, 128, bs,
                                               8, None, None)


def _decode(pa, stride, B=3, bs=16):
    return pa.lib.pa_decode_attention_q8_strided(A, A, A, A, A, A, A, 4, A, stride, B, 64, 8, 2, 128,
                                                 bs, 16, 0.1, None, 0, None, None)


def _prefill(pa, stride, T=10, bs=16):
    return pa.lib.pa_prefill_attention_q8_strided(A, A, A, T, 8, A, A, A, A, A, 4, A, stride, 2, 64,
                                                  8, 2, 128, bs, 32, 0.1, None, None)


@pytest.mark.parametrize("call", [_append, _decode, _prefill])
def test_refusals(pa, call):
    assert call(pa, -1) == pa.PA_ERR_INVALID_ARG
    assert call(pa, 2, bs=8) == pa.PA_ERR_UNSUPPORTED


def test_nothing_to_do(pa):
    assert _append(pa, 2, T=0) == 0 and _decode(pa, 2, B=0) == 0 and _prefill(pa, 0, T=0) == 0


def test_bindings_check_the_lengths(pa):
    # (the one thing about them that a CPU can show: kind and shape)
    tab = torch.zeros(3, 2, dtype=torch.int32)
    lens = torch.zeros(3, 2, dtype=torch.int32)[:, 0]
    assert pa._tables(tab, lens, 3) == (2, 2)
    assert pa._tables(tab, lens[:1].expand(3), 3) == (2, 0)
    for bad in (lens.long(), lens[:2], torch.zeros(3, 1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            pa._tables(tab, bad, 3)
