"""Writes to and read-back from a paged key/value cache vs the fp64 oracle (GPU).

bf16 rows without rotation are copies; rotated rows follow tests/test_gpu_rope_apply.py.  E4M3: the
scale is amax / 448 in fp32 (one rounding, 2^-24; rotated values add 2^-21 of the pair's
magnitudes), codes are the oracle's except where its quotient lies within the fp32 error of a
rounding midpoint (tests.helpers.check_codes: 2^-22 relative unrotated, rotated 2^-19 of the
largest quotient 448, the pair sum being at most twice the row's largest value).
"""

import numpy as np
import pytest
import torch

from exact_attention_46_gb300 import _lib, ops, synth
from oracle import e4m3, paged
from tests.helpers import check_codes, to64
from tests.test_gpu_rope_apply import check as check_rope

pytestmark = pytest.mark.gpu


def draw(shape, case, stream):
    return torch.from_numpy(synth.normal(shape, synth.seed_for(case, stream))).to(torch.bfloat16)


def new_cache(n_pages, Hkv, page, D, fp8, token_major, fill=0x35):
    shape = (n_pages, page, Hkv, D) if token_major else (n_pages, Hkv, page, D)
    if fp8:
        kv = [torch.full(shape, fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
        sc = [torch.full((n_pages, Hkv, page), 3.25, device="cuda") for _ in range(2)]
        return kv, sc
    return [torch.full(shape, 0.71875, dtype=torch.bfloat16, device="cuda") for _ in range(2)], [None, None]


def rows_of(cache, slots, page, token_major):
    """[tokens, Hkv, D] rows of the cache at the slots, on the CPU."""
    c = cache.cpu() if token_major else cache.cpu().transpose(1, 2)
    return c[slots // page, slots % page]


def scales_of(scale, slots, page):
    return scale.cpu().transpose(1, 2)[slots // page, slots % page]


CASES = [(1, 1, 1, 64, 16, False), (5, 8, 2, 128, 32, True), (130, 6, 6, 64, 16, True), (77, 4, 1, 256, 128, False),
         (300, 12, 3, 128, 64, False), (9, 5, 5, 256, 1024, True)]


@pytest.mark.parametrize("T,Hq,Hkv,D,page,token_major", CASES)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("turn", [None, "interleaved", "half"])
def test_append_matches_oracle(T, Hq, Hkv, D, page, token_major, fp8, turn):
    rng = np.random.default_rng(T + D)
    qkv = draw((T, Hq + 2 * Hkv, D), 140, 0)
    if T > 3:
        qkv[2] = 0                                      # a token of zeros
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    n_pages = (T + page - 1) // page + 2
    slots = torch.from_numpy(rng.permutation(n_pages * page)[:T].astype(np.int64))
    pad = torch.from_numpy(rng.random(T) < 0.2)
    given = torch.where(pad, torch.tensor(-1 - 5 * T), slots)
    (kc, vc), (ks, vs) = new_cache(n_pages, Hkv, page, D, fp8, token_major)
    before = [t.clone() for t in (kc, vc, ks, vs) if t is not None]
    dev = qkv.cuda()
    dq, dk, dv = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    k_ref, gain, rot = to64(k), 1.0, 0
    if turn is None:
        ops.kv_cache_append(dk, dv, kc, vc, given.cuda(), ks, vs, token_major=token_major)
    else:
        rot, half = D // 2, turn == "half"
        pos = rng.integers(0, 3000, T).astype(np.int32)
        cs = ops.rope_scaled_table(3000, rot, scaling="yarn", factor=4.0, original_length=700)
        q_out = ops.rope_kv_cache_append(dq, dk, dv, cs, torch.from_numpy(pos).cuda(), kc, vc, given.cuda(), ks, vs,
                                         half=half, token_major=token_major)
        th, gain = paged.frequencies(rot, 10000.0, "yarn", 4.0, 700.0)
        k_ref = paged.rotate(to64(k), pos, th, gain, half)
        check_rope(q_out, to64(q), paged.rotate(to64(q), pos, th, gain, half), rot, half, gain)
    ops.check()
    live = slots[~pad]
    if fp8:
        for cache, scale, ref, turned in ((kc, ks, k_ref[~pad.numpy()], turn is not None), (vc, vs, to64(v)[~pad.numpy()], False)):
            if len(ref) == 0:
                continue
            codes, s, pre = paged.quantise_rows(ref)
            np.testing.assert_allclose(scales_of(scale, live, page).double().numpy(), s, rtol=2.0 ** -19 if turned else 2.0 ** -23)
            check_codes(rows_of(cache, live, page, token_major).numpy(), {"codes": codes, "pre": pre}, 2.0 ** -22,
                        448 * 2.0 ** -19 if turned else 0.0)
    else:
        got = rows_of(kc, live, page, token_major)
        if turn is None:
            assert torch.equal(got, k[~pad])
        else:
            check_rope(got, to64(k)[~pad.numpy()], k_ref[~pad.numpy()], rot, turn == "half", gain)
        assert torch.equal(rows_of(vc, live, page, token_major), v[~pad])
    # every other row is as it was
    untouched = torch.ones(n_pages * page, dtype=torch.bool)
    untouched[live] = False
    rest = torch.nonzero(untouched).flatten()
    for t, b in zip([x for x in (kc, vc, ks, vs) if x is not None], before):
        if t.dim() == 4:
            assert torch.equal(rows_of(t, rest, page, token_major), rows_of(b, rest, page, token_major))
        else:
            assert torch.equal(scales_of(t, rest, page), scales_of(b, rest, page))


def test_codes_are_those_of_the_fp32_quotient():
    # unrotated rows of very different sizes: scale and codes are bit for bit amax / 448 and the E4M3
    # rounding of x / scale in fp32 (torch's division -- by a tensor: by a number it multiplies with a
    # rounded reciprocal -- and cast)
    T, H, D, page = 4096, 4, 128, 64
    x = synth.normal((T, H, D), synth.seed_for(145, 0)) * np.exp2(np.random.default_rng(9).uniform(-90, 90, (T, H, 1)))
    k = torch.from_numpy(x).to(torch.bfloat16).cuda()
    (kc, vc), (ks, vs) = new_cache(T // page, H, page, D, True, False)
    ops.kv_cache_append(k, k, kc, vc, torch.arange(T, device="cuda"), ks, vs)
    ops.check()
    amax = k.float().abs().amax(-1)
    scale = amax / torch.full_like(amax, 448.0)
    codes = (k.float() / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(ks.transpose(1, 2).reshape(T, H), scale)
    assert torch.equal(kc.transpose(1, 2).reshape(T, H, D), codes)


def test_rows_that_are_not_finite_or_tiny():
    D, page = 64, 16
    k = torch.ones((4, 1, D), dtype=torch.bfloat16)
    k[0, 0, 5] = float("nan")
    k[1, 0, 6] = float("inf")
    k[2] = 2.0 ** -126                                 # a scale below the smallest normal fp32
    (kc, vc), (ks, vs) = new_cache(1, 1, page, D, True, False)
    ops.kv_cache_append(k.cuda(), k.cuda(), kc, vc, torch.arange(4, device="cuda"), ks, vs)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    ko, vo = ops.kv_cache_gather(kc, vc, table, cu, 4, ks, vs)
    ops.check()
    for o in (ko, vo):
        assert torch.isnan(o[:2]).all() and torch.all(o[2] == 0)
        # amax / 448 rounds once, code 448 times it: within an fp32 step of 1
        assert torch.all((o[3].float() - 1).abs() <= 2.0 ** -8)
    assert ks[0, 0, 2] == 1


def test_slots_past_the_cache_are_reported_and_not_written():
    (kc, vc), _ = new_cache(2, 3, 16, 64, False, True)
    k, v = draw((4, 3, 64), 141, 0).cuda(), draw((4, 3, 64), 141, 1).cuda()
    before = kc.clone()
    ops.kv_cache_append(k, v, kc, vc, torch.tensor([32, 1 << 40, -7, 31], device="cuda"), token_major=True)
    with pytest.raises(_lib.AttnError, match="slot"):
        ops.check()
    assert torch.equal(kc.view(32, 3, 64)[:31], before.view(32, 3, 64)[:31]) and torch.equal(kc.view(32, 3, 64)[31], k[3])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("lens,page,Hkv,D", [([1], 16, 1, 64), ([5, 0, 300, 17, 64, 0], 16, 5, 128), ([129, 1000], 256, 2, 256),
                                             ([33] * 40, 32, 8, 64)])
def test_gather_matches_rows(lens, page, Hkv, D, token_major, fp8):
    rng = np.random.default_rng(len(lens))
    need = [(n + page - 1) // page for n in lens]
    n_pages = sum(need) + 1
    (kc, vc), (ks, vs) = new_cache(n_pages, Hkv, page, D, fp8, token_major)
    for i, c in enumerate((kc, vc)):
        if fp8:
            codes = torch.from_numpy(rng.integers(0, 256, tuple(c.shape)).astype(np.uint8))
            codes[(codes & 0x7F) == 0x7F] = 0
            c.copy_(codes)
            (ks, vs)[i].copy_(torch.from_numpy(np.exp2(rng.uniform(-8, 8, tuple(ks.shape))).astype(np.float32)))
        else:
            c.copy_(draw(tuple(c.shape), 142, i))
    table = np.full((len(lens), max(need) + 2), 1 << 30, np.int32)     # unused entries are not read
    perm, at = rng.permutation(n_pages), 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    ko, vo = ops.kv_cache_gather(kc, vc, torch.from_numpy(table).cuda(), torch.from_numpy(cu).cuda(), int(cu[-1]), ks, vs,
                                 token_major=token_major)
    ops.check()
    slots = torch.from_numpy(np.concatenate([table[s, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
                                             for s, n in enumerate(lens)]))
    for out, c, sc in ((ko, kc, ks), (vo, vc, vs)):
        rows = rows_of(c, slots, page, token_major)
        if not fp8:
            assert torch.equal(out.cpu(), rows)
        else:
            ref = e4m3.decode(rows.numpy()) * scales_of(sc, slots, page).double().numpy()[..., None]
            # the fp32 product is exact to 2^-24, then one rounding to bf16
            assert np.all(np.abs(to64(out) - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref))


def test_gather_reports_rows_it_cannot_place():
    (kc, vc), _ = new_cache(3, 2, 16, 64, False, False)
    kc.copy_(draw(tuple(kc.shape), 143, 0))
    table = torch.tensor([[0, 9], [-1, 2]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 20, 24], dtype=torch.int32, device="cuda")   # rows 16.. of 0 in page 9, 1 in page -1
    ko = torch.full((26, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    ops.kv_cache_gather(kc, vc, table, cu, 26, k_out=ko, v_out=vo)     # and two rows past the last sequence
    with pytest.raises(_lib.AttnError, match="sequence or page"):
        ops.check()
    assert torch.equal(ko[:16], kc[0].transpose(0, 1)) and torch.all(ko[16:] == 7.0) and torch.all(vo[16:] == 7.0)


def test_rows_beyond_four_gigabytes():
    # 2^32 elements and more before the last page: 64-bit offsets in the write and the read
    Hkv, page, D = 8, 1024, 256
    n_pages = 2 ** 32 // (Hkv * page * D) + 2
    if torch.cuda.mem_get_info()[0] < 3 * n_pages * Hkv * page * D * 2:
        pytest.skip("not enough device memory")
    kc, vc = (torch.empty((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = draw((3, Hkv, D), 144, 0).cuda(), draw((3, Hkv, D), 144, 1).cuda()
    at = torch.tensor([n_pages * page - 3, n_pages * page - 2, n_pages * page - 1], device="cuda")
    ops.kv_cache_append(k, v, kc, vc, at)
    assert torch.equal(kc[-1, :, -3:].transpose(0, 1), k)
    table = torch.full((1, 1), n_pages - 1, dtype=torch.int32, device="cuda")
    ko, vo = ops.kv_cache_gather(kc, vc, table, torch.tensor([0, 1024], dtype=torch.int32, device="cuda"), 1024)
    ops.check()
    assert torch.equal(ko[-3:], k) and torch.equal(vo[-3:], v)
