"""Rotary positions on their own (rope_apply, rope_scaled_table) vs the fp64 oracle (GPU).

Tolerance: the table holds fp32 (cos, sin), each off by half an fp32 step (2^-24 relative to at
most the multiplier, plus the fp64 angle's own last bits); the turn adds two products and a sum
in fp32 (3 * 2^-24 of |x_a| + |x_b|), and the output rounds once to bf16 (half a step, 2^-8 of the
value).  So |err| <= 2^-8 |y| + 2^-21 gain (|x_a| + |x_b|), the second term with a factor to spare.
"""

import numpy as np
import pytest
import torch

from exact_attention_46_gb300 import _lib, ops, synth
from oracle import paged
from tests.helpers import to64

pytestmark = pytest.mark.gpu

SCALED = [("none", 1.0, 0.0), ("linear", 4.0, 0.0), ("ntk", 8.0, 0.0), ("yarn", 16.0, 2048.0)]


def draw(shape, case):
    return torch.from_numpy(synth.normal(shape, synth.seed_for(case, synth.STREAM_Q))).to(torch.bfloat16)


def pair_sum(x, rot, half):
    """|x_a| + |x_b| of each element's pair (the element itself past rot)."""
    a = np.abs(x).copy()
    at = np.arange(rot // 2) if half else np.arange(0, rot, 2)
    bt = at + rot // 2 if half else at + 1
    s = a[..., at] + a[..., bt]
    a[..., at] = s
    a[..., bt] = s
    return a


def check(got, x, ref, rot, half, gain):
    err = np.abs(to64(got) - ref)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * gain * pair_sum(x, rot, half)
    assert np.all(err <= tol), float((err - tol).max())


@pytest.mark.parametrize("scaling,factor,length", SCALED)
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_scaled_table_matches_oracle(scaling, factor, length, rot):
    n = 40000
    cs = ops.rope_scaled_table(n, rot, 10000.0, scaling, factor, length)
    ops.check()
    th, gain = paged.frequencies(rot, 10000.0, scaling, factor, length)
    ang = np.arange(n)[:, None] * th[None]
    ref = gain * np.stack([np.cos(ang), np.sin(ang)], -1)
    # half an fp32 step, and the fp64 frequencies' last bits at angles up to 4e4
    assert np.abs(to64(cs) - ref).max() <= gain * (2.0 ** -24 + 4e4 * 2.0 ** -50)


def test_unscaled_table_is_the_cos_sin_table():
    assert torch.equal(ops.rope_scaled_table(3000, 128, 10000.0), ops.rope_cos_sin_table(3000, 128, 10000.0))


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 112), (256, 256), (256, 64)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
def test_matches_oracle(D, rot, half, transpose):
    for i, (T, H) in enumerate([(1, 1), (7, 3), (130, 4), (33, 9)]):
        scaling, factor, length = SCALED[(i + rot // 16) % 4]
        x = draw((T, H, D), 100 + i)
        pos = np.random.default_rng(i).integers(0, 5000, T).astype(np.int32)
        cs = ops.rope_scaled_table(5000, rot, 10000.0, scaling, factor, length)
        got = ops.rope_apply(x.cuda(), cs, torch.from_numpy(pos).cuda(), half=half, transpose=transpose)
        ops.check()
        th, gain = paged.frequencies(rot, 10000.0, scaling, factor, length)
        check(got, to64(x), paged.rotate(to64(x), pos, th, gain, half, transpose), rot, half, gain)


@pytest.mark.parametrize("half", [False, True])
def test_gradient_against_differences(half):
    # a linear map: the directional difference of the kernel's forward, on inputs x +- e, times dy
    # equals e times the kernel's gradient; the bf16 roundings (2^-8 of |y| or |dx| each, summed
    # over the elements) bound the gap
    T, H, D = 40, 3, 128
    x, e, dy = (draw((T, H, D), 120 + i).cuda() for i in range(3))
    cs = ops.rope_scaled_table(64, 64, scaling="yarn", factor=8.0, original_length=16)
    fwd = [to64(ops.rope_apply((x.float() + s * e.float()).to(torch.bfloat16), cs, half=half)) for s in (1, -1)]
    dx = ops.rope_apply(dy, cs, half=half, transpose=True)
    ops.check()
    step = (to64((x.float() + e.float()).to(torch.bfloat16)) - to64((x.float() - e.float()).to(torch.bfloat16))) / 2
    gap = ((fwd[0] - fwd[1]) / 2 * to64(dy)).sum() - (step * to64(dx)).sum()
    bound = 2.0 ** -8 * ((np.abs(fwd[0]) + np.abs(fwd[1])) / 2 * np.abs(to64(dy)) + np.abs(step * to64(dx))).sum()
    assert abs(gap) <= bound
    # and far inside the bound if the roundings are independent: their sum grows with the root
    assert abs(gap) <= 8 * bound / np.sqrt(T * H * D)


def test_positions_default_to_the_token_index():
    x = draw((2, 50, 4, 64), 130).cuda()
    cs = ops.rope_scaled_table(64, 64)
    pos = torch.arange(50, dtype=torch.int32, device="cuda").expand(2, 50).contiguous()
    assert torch.equal(ops.rope_apply(x, cs), ops.rope_apply(x, cs, pos))


def test_views_in_place_and_streams():
    qkv = draw((37, 12, 128), 131).cuda()
    cs = ops.rope_scaled_table(64, 128)
    q, k = qkv[:, :8], qkv[:, 8:10]
    want_q, want_k = ops.rope_apply(q.contiguous(), cs), ops.rope_apply(k.contiguous(), cs)
    rest = qkv[:, 10:].clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ops.rope_apply(q, cs, out=q, stream=st)            # in place, on a view, on another stream
    got_k = ops.rope_apply(k, cs, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    ops.check()
    assert torch.equal(q, want_q) and torch.equal(got_k, want_k) and torch.equal(qkv[:, 10:], rest)


def test_a_position_outside_the_table_is_reported_and_not_written():
    x = draw((4, 2, 64), 132).cuda()
    cs = ops.rope_scaled_table(10, 64)
    out = torch.full_like(x, 7.0)
    ops.rope_apply(x, cs, torch.tensor([3, 10, -1, 9], dtype=torch.int32, device="cuda"), out=out)
    with pytest.raises(_lib.AttnError, match="position"):
        ops.check()
    assert torch.all(out[1:3] == 7.0)
    ok = ops.rope_apply(x[[0, 3]], cs, torch.tensor([3, 9], dtype=torch.int32, device="cuda"))
    assert torch.equal(out[[0, 3]], ok)
    ops.check()
