"""Sizes and boundaries past 31 bits are refused before the call: the library takes them as C ints, and ctypes would hand it
their low 32 bits (2^32 rows would be none, a row of 2^32 + 128 channels one of 128). Tensors without memory, so no GPU."""
import pytest
import torch

import rotated_w4a8_group_amd as pq

WRAP = 2 ** 32
F16, U8, F32, I32 = torch.float16, torch.uint8, torch.float32, torch.int32


def _e(*shape, dtype=F16):
    return torch.empty(shape, dtype=dtype, device="meta")


def _layer(K, N):
    """Packed weights of the low 32 bits of K and N, which is what the library would be asked for, and the whole size's sz."""
    return _e(pq.lib().pq_packed_weight_bytes(K % WRAP, N % WRAP), dtype=U8), _e(K // 128, N, 2)


def _codes(M, K, dtype=U8):
    return _e(1, M, K, dtype=dtype), _e(1, M, K // 128, dtype=F32), _e(1, M, K // 128, dtype=F32)


BIG_K, BIG_N = WRAP + 128, WRAP + 64
CALLS = {
    "block_norms rows": lambda: pq.block_norms(_e(WRAP, 8), _e(WRAP, 8)),
    "block_norms rows, one too many": lambda: pq.block_norms(_e(2 ** 31, 8), _e(2 ** 31, 8)),
    "block_norms channels": lambda: pq.block_norms(_e(1, WRAP + 8), _e(1, WRAP + 8)),
    "rotate rows": lambda: pq.rotate(_e(WRAP, 128), _e(8, 64, 8, dtype=U8), _e(128)),
    "rotate channels": lambda: pq.rotate(_e(1, BIG_K), _e(8, BIG_K // 2, 8, dtype=U8), _e(BIG_K)),
    "rotate_quant channels": lambda: pq.rotate_quant(_e(1, BIG_K), _e(8, BIG_K // 2, 8, dtype=U8), _e(BIG_K)),
    "rotate_quant_tok rows": lambda: pq.rotate_quant_tok(_e(WRAP, 128), _e(8, 64, 8, dtype=U8), _e(128)),
    "add_rms_rotate_quant rows": lambda: pq.add_rms_rotate_quant(_e(WRAP, 128), _e(WRAP, 128), _e(128), 1e-6, _e(8, 64, 8, dtype=U8), _e(128)),
    "matvec channels": lambda: pq.matvec(_e(1, BIG_K), *_layer(BIG_K, 64), 64),
    "matvec columns": lambda: pq.matvec(_e(1, 128), *_layer(128, BIG_N), BIG_N),
    "matvec boundary": lambda: pq.matvec(_e(2, 1, 128), *_layer(128, 256), 256, BIG_K),
    "matvec second boundary": lambda: pq.matvec(_e(3, 1, 128), *_layer(128, 384), 384, 128, BIG_K + 128),
    "matvec boundary below": lambda: pq.matvec(_e(2, 1, 128), *_layer(128, 256), 256, 128 - WRAP),
    "gemm_glu rows": lambda: pq.gemm_glu(*_codes(WRAP, 128), *_layer(128, 32), 16),
    "gemm_glu channels": lambda: pq.gemm_glu(*_codes(1, BIG_K), *_layer(BIG_K, 32), 16),
    "gemm_glu columns": lambda: pq.gemm_glu(*_codes(1, 128), *_layer(128, WRAP + 32), 2 ** 31 + 16),
    "gemm rows": lambda: pq.gemm(*_codes(WRAP, 128), *_layer(128, 32), 32),
    "gemm channels": lambda: pq.gemm(*_codes(1, BIG_K), *_layer(BIG_K, 32), 32),
    "gemm boundary": lambda: pq.gemm(*_codes(1, 128), *_layer(128, 256), 256, WRAP),
    "gemm_prepared columns": lambda: pq.gemm_prepared(*_codes(1, 128), *_layer(128, BIG_N), BIG_N),
    "gemm_i8 channels": lambda: pq.gemm_i8(*_codes(1, BIG_K, torch.int8), *_layer(BIG_K, 32), 32),
    "gemm_noalloc columns": lambda: pq.gemm_noalloc(*_codes(1, 128), *_layer(128, BIG_N), BIG_N, out=_e(1, BIG_N, dtype=torch.bfloat16)),
    "pack_weights channels": lambda: pq.pack_weights(_e(BIG_K, 2, dtype=I32), _e(BIG_K // 128, 2, dtype=I32), _e(BIG_K // 128, 16)),
    "pack_weights5 columns": lambda: pq.pack_weights5(_e(128, WRAP // 8, dtype=I32), _e(128, WRAP // 32, dtype=I32), _e(1, WRAP // 8, dtype=I32),
                                                      _e(1, WRAP // 32, dtype=I32), _e(1, WRAP)),
    "workspace of a gemm": lambda: pq.gemm_workspace_bytes(WRAP + 40, 256, 128),
    "workspace of a gemm_tok": lambda: pq.gemm_tok_workspace_bytes(40, 256, BIG_K),
}


@pytest.mark.parametrize("name", CALLS)
def test_refused(name):
    with pytest.raises(ValueError, match="at most 2\\^31 - 1 in one call"):
        CALLS[name]()


def test_no_boundary_and_past_the_columns_are_taken():
    """The largest int is still 'no boundary', in either place: the call gets as far as its tensors' device."""
    for pb in ((), (pq.NO_BOUNDARY,), (pq.NO_BOUNDARY, pq.NO_BOUNDARY), (4096, pq.NO_BOUNDARY)):
        with pytest.raises(TypeError, match="CUDA"):
            pq.matvec(_e(1, 128), *_layer(128, 256), 256, *pb)
        with pytest.raises(TypeError, match="CUDA"):
            pq.gemm(*_codes(1, 128), *_layer(128, 256), 256, *pb)


@pytest.mark.parametrize("M,K,F,P", [(2 ** 20 + 1, 128, 65536, 1), (2 ** 21, 256, 32784, 1), (2 ** 23, 128, 2 ** 16, 2), (2 ** 20 - 128, 2048, 2 ** 18, 1)])
def test_gemm_glu_of_more_threads_than_a_launch_counts(M, K, F, P):
    """Refused before the pass over the scales is queued (no address is real, so nothing may be launched)."""
    at = [(1 << 44) + (i << 40) for i in range(7)]
    rc = pq.lib().pq_gemm_glu(at[0], at[1], at[2], M, K, P, at[3], at[4], F, 0, at[5], F, 0, at[6], 1 << 40, 0, None)
    assert rc == -2 and b"too many for one call" in pq.lib().pq_last_error()
