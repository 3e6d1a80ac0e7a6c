"""The entry points of rotary positions and the paged cache reject bad arguments before touching
the device (CPU only), through the C ABI and the Python binding."""

import pytest
import torch

import tests.test_abi as abi
from exact_attention_46_gb300 import ops

lib = abi.lib
F = 1 << 24          # 16-byte aligned non-null fake device addresses, 16 MB apart: never dereferenced


def sweep(f, ok, cases):
    for i, val, code in cases:
        a = list(ok)
        a[i] = val
        assert f(*a) == code, (i, val)


def test_scaled_table(lib):
    ok = [F, 4096, 64, 10000.0, 3, 4.0, 1024.0, None]
    sweep(lib.rope_scaled_table, ok, [(0, None, 1), (0, F + 4, 1), (1, 0, 1), (1, (1 << 26) + 1, 1), (2, 63, 1), (2, 2, 1),
                                      (3, 0.0, 1), (3, float("inf"), 1), (4, 4, 1), (4, -1, 1), (5, 0.5, 1),
                                      (5, float("nan"), 1), (6, 0.0, 1)])


def test_rope_apply(lib):
    #     x  out    cs     pos  n  seq H  D    xs   os   n_pos rot lay tr stream
    ok = [F, F * 2, F * 3, F * 4, 9, 0, 4, 128, 512, 512, 4096, 64, 0, 0, None]
    sweep(lib.rope_apply, ok, [
        (0, None, 1), (0, F + 8, 1), (1, F + 512, 1), (2, None, 1), (2, F * 3 + 4, 1), (3, F * 4 + 2, 1), (4, 0, 1),
        (6, 0, 1), (7, 96, 2), (7, 0, 1), (8, 511, 1), (8, 516, 1), (8, 256, 1), (9, 256, 1), (10, 0, 1), (11, 8, 1),
        (11, 72, 1), (11, 144, 1), (12, 2, 1), (13, 2, 1), (1, F * 3, 1)])
    no_pos = list(ok)
    no_pos[3] = None                                   # seq_len 0 without positions
    assert lib.rope_apply(*no_pos) == 1
    no_pos[5] = 4097                                   # longer than the table
    assert lib.rope_apply(*no_pos) == 1
    shifted = list(ok)
    shifted[1] = F                                     # in place, but with another stride
    shifted[9] = 1024
    assert lib.rope_apply(*shifted) == 1


def test_append(lib):
    #     k  v      kc     vc     ks     vs     slots  n  Hkv D    kst  vst  pages page lay dt stream
    ok = [F, F * 2, F * 3, F * 4, F * 5, F * 6, F * 7, 9, 4, 128, 512, 512, 10, 64, 0, 1, None]
    sweep(lib.kv_cache_append, ok, [
        (0, None, 1), (1, F * 2 + 8, 1), (2, None, 1), (3, F * 3 + 16, 1), (4, None, 1), (5, None, 1), (4, F * 5 + 4, 1),
        (6, None, 1), (6, F * 7 + 4, 1), (7, 0, 1), (8, 0, 1), (9, 96, 2), (10, 256, 1), (11, 513, 1), (12, 0, 1),
        (13, 0, 1), (13, 48, 2), (13, 8, 2), (13, 2048, 2), (14, 2, 1), (15, 2, 1),
        (15, 0, 1),                                    # bf16 with scales
        (2, F, 1),                                     # cache over k
        (4, F * 7, 1)])                                # scales over slots
    # q  k  v  q_out  cs  pos  kc  vc  ks  vs  slots  n  Hq Hkv D  qs  ks  vs  pages page lay dt n_pos rot rl stream
    ok = [F, F * 2, F * 3, F * 4, F * 5, F * 6, F * 7, F * 8, None, None, F * 9, 9, 8, 4, 128, 1024, 512, 512, 10, 64, 1, 0,
          4096, 128, 1, None]
    sweep(lib.rope_kv_cache_append, ok, [
        (0, None, 1), (3, None, 1), (4, None, 1), (5, None, 1), (5, F * 6 + 2, 1), (12, 0, 1), (15, 512, 1), (22, 0, 1),
        (23, 136, 1), (24, 3, 1), (3, F * 7, 1), (8, F * 10, 1)])


def test_gather(lib):
    #     kc vc     ks     vs     table  cu     ko     vo     n  tot Hkv D  pages page maxp lay dt stream
    ok = [F, F * 2, F * 3, F * 4, F * 5, F * 6, F * 7, F * 8, 3, 100, 4, 128, 10, 64, 2, 0, 1, None]
    sweep(lib.kv_cache_gather, ok, [
        (0, None, 1), (2, None, 1), (4, None, 1), (4, F * 5 + 2, 1), (5, None, 1), (6, None, 1), (7, F * 8 + 8, 1), (8, 0, 1),
        (9, 0, 1), (10, 0, 1), (11, 96, 2), (12, 0, 1), (13, 100, 2), (14, 0, 1), (15, 5, 1), (16, 0, 1), (6, F, 1), (7, F * 7, 1)])


def test_attention(lib):
    ws = lib.attn_decode_paged_workspace_bytes(3, 4, 8, 2, 128, 64, 5)
    assert ws > 0
    assert lib.attn_decode_paged_workspace_bytes(3, 4, 8, 2, 128, 64, 2) == 0       # one tile: no merge
    for bad in ((0, 4, 8, 2, 128, 64, 5), (3, 65, 8, 2, 128, 64, 5), (3, 4, 7, 2, 128, 64, 5), (3, 4, 8, 2, 96, 64, 5)):
        assert lib.attn_decode_paged_workspace_bytes(*bad) == 0
    # q kc vc ks vs o lse table ctx ql mask ws bytes B T Hq Hkv D pages page maxp lay dt scale stream
    ok = [F, F * 2, F * 3, F * 4, F * 5, F * 6, F * 7, F * 8, F * 9, F * 10, F * 11, F * 12, ws, 3, 4, 8, 2, 128, 20, 64, 5, 0,
          1, 0.0, None]
    sweep(lib.attn_decode_paged, ok, [
        (0, None, 1), (1, None, 1), (3, None, 1), (5, F * 6 + 8, 1), (6, F * 7 + 2, 1), (7, None, 1), (8, None, 1),
        (9, F * 10 + 1, 1), (10, F * 11 + 4, 1), (11, None, 1), (11, F * 12 + 8, 1), (12, ws - 1, 1), (13, 0, 1), (13, 1025, 2),
        (14, 0, 1), (14, 65, 2), (15, 7, 1), (15, 0, 1), (16, 0, 1), (17, 256, 2), (17, 96, 2), (18, 0, 1), (19, 24, 2),
        (20, 0, 1), (20, 1 << 26, 1), (21, 2, 1), (22, 0, 1), (22, 3, 1), (23, -1.0, 1), (23, float("nan"), 1),
        (5, F, 1), (6, F * 2, 1), (11, F * 6, 1), (5, F * 9, 1)])


def test_binding_checks_come_first():
    bf, f32 = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 4, 64))
    with pytest.raises(ValueError, match="dtype"):
        ops.rope_apply(f32, None)
    with pytest.raises(ValueError, match="dimensions"):
        ops.rope_apply(bf[0], None)
    with pytest.raises(ValueError, match="contiguous"):
        ops.rope_apply(bf.transpose(1, 2), None)
    with pytest.raises(ValueError, match="CUDA"):
        ops.rope_apply(bf, None)
    with pytest.raises(ValueError, match="CUDA"):
        ops.kv_cache_append(bf, bf, bf, bf, None)
    with pytest.raises(ValueError, match="evenly"):
        ops.rope_apply(torch.zeros((2, 9, 4, 64), dtype=torch.bfloat16)[:, :5], None)
    with pytest.raises(ValueError, match="dimensions"):
        ops.kv_cache_gather(bf, bf, None, None, 1)
    with pytest.raises(ValueError, match="dtype"):
        ops.attn_decode_paged(f32[None], bf, bf, None, None)
    with pytest.raises(ValueError, match="scaling"):
        ops.rope_scaled_table(8, 64, scaling="cubic")
    with pytest.raises(TypeError):
        ops.rope_apply([1], None)
