"""Attention of single and tree-drafted tokens over a paged cache (attn_decode_paged) vs the fp64
oracle, through the C ABI (GPU).

Both sides read the same cache bytes.  Error bound per output element, from the kernel's
roundings: with X = max_j scale sum_d |q_d k_jd| over the seen keys and A = sum_j p_j |v_j|,
* a logit is a D-term fp32 sum of exact products times fp32 constants: off by at most
  dx = (D + 16) 2^-24 X; the probabilities then by a factor 1 +- 2 dx, and exp2's own 2^-22;
* a numerator rounds to bf16 (half a step, 2^-8 of it) or, over an E4M3 cache, to fp16 (2^-11; the
  scaled numerators' subnormal step adds less than 2^-26 of the largest value scale per key);
* the output rounds to bf16: 2^-8 of it.
So |err| <= 2^-8 |o| + (r + 2 dx + 2^-18) A (+ L 2^-26 448 max scale), r = 2^-8 or 2^-11, and
|lse err| <= dx + 2^-18 (1 + |lse|).
Over an E4M3 cache with more than 8 rows (group x drafts) the products run on E4M3 terms:
* a query row, scaled so that its largest element lies in [128, 256), is the sum of two terms.  An
  element of eight significant bits leaves a remainder of four after the first term, which the
  second holds exactly unless it lies below E4M3's smallest step 2^-9: that is off by at most half
  a step, 2^-10, so by 2^-17 of the row's largest element (and only in elements below 2^-9 of
  it).  A logit moves by at most 2^-17 scale max|q| sum_d |k_jd| more;
* a numerator times its value's scale over 2^-11 vref (vref a power of two, at most twice the largest
  scale) is rounded to fp16 (2^-11) and to the sum of three E5M2 terms: each of the first two cuts three
  bits off the top and the third rounds to three, 2^-9 of the number in all, or half of E5M2's smallest
  step, 2^-17, where that is more: 2^-27 of the largest scale times the value's code, per key, over a sum
  of at least 1.  So r = 2^-9 + 2^-11, and the last term (2^-26 448 max scale a key) covers the rest.
What no row may see -- free rows of used pages, free pages, entries behind the page table's end -- holds
NaN.
"""

import numpy as np
import pytest
import torch

from exact_attention_46_gb300 import _lib, ops, synth
from oracle import e4m3, paged
from tests.helpers import to64

pytestmark = pytest.mark.gpu


class Problem:
    """Random sequences in a paged cache whose unused bytes are NaN."""

    def __init__(self, ctx, T, Hq, Hkv, D, page, fp8=False, token_major=False, tree=False, q_lens=None, case=150,
                 gain=1.0, extra_pages=2):
        self.ctx, self.T, self.Hq, self.Hkv, self.D, self.page = list(ctx), T, Hq, Hkv, D, page
        self.fp8, self.token_major = fp8, token_major
        B = self.B = len(ctx)
        rng = self.rng = np.random.default_rng(case)
        self.ql = list(q_lens) if q_lens is not None else [T] * B
        self.given_ql = q_lens is not None
        self.L = [c + q for c, q in zip(self.ctx, self.ql)]
        need = [(n + page - 1) // page for n in self.L]
        self.n_pages = sum(need) + extra_pages
        self.max_pages = max(1, max(need)) + 1
        self.table = np.full((B, self.max_pages), -12345, np.int32)
        perm, at = rng.permutation(self.n_pages), 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.q = torch.from_numpy(synth.normal((B, T, Hq, D), synth.seed_for(case, 0)) * gain).to(torch.bfloat16)
        shape = (self.n_pages, Hkv, page, D)
        self.cache, self.scale, self.val = [], [], []
        used = np.zeros((self.n_pages, page), bool)
        for b in range(B):
            j = np.arange(self.L[b])
            used[self.table[b, j // page], j % page] = True
        hidden = ~np.broadcast_to(used[:, None], shape[:3])
        for i in range(2):
            x = synth.normal(shape, synth.seed_for(case, 1 + i))
            x = x * np.exp2(rng.uniform(-3, 3, shape[:3]))[..., None]
            if fp8:
                codes, s, _ = paged.quantise_rows(x)
                s = s.astype(np.float32)
                codes[hidden] = 0x7F
                s[hidden] = np.nan
                val = e4m3.decode(codes) * s.astype(np.float64)[..., None]
                c = torch.from_numpy(codes)
                self.scale.append(torch.from_numpy(s).cuda())
            else:
                x[hidden] = np.nan
                c = torch.from_numpy(x).to(torch.bfloat16)
                val = to64(c)
                self.scale.append(None)
            self.val.append(val)
            self.cache.append((c.transpose(1, 2).contiguous() if token_major else c).cuda())
        self.mask = None
        if tree:
            self.mask = np.zeros((B, T), np.uint64)
            for b in range(B):
                for t in range(T):
                    up = int(rng.integers(max(0, t - 5) - 1, t))
                    self.mask[b, t] = (self.mask[b, up] if up >= 0 else np.uint64(0)) | (np.uint64(1) << np.uint64(t))

    def args(self):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        kw = dict(k_scale=self.scale[0], v_scale=self.scale[1], token_major=self.token_major,
                  q_lens=dev(np.array(self.ql, np.int32)) if self.given_ql else None,
                  tree_mask=dev(self.mask.view(np.int64)) if self.mask is not None else None)
        return (self.q.cuda(), self.cache[0], self.cache[1], dev(self.table), dev(np.array(self.ctx, np.int32))), kw

    def rows(self, i, b):
        j = np.arange(self.L[b])
        return self.val[i].transpose(0, 2, 1, 3)[self.table[b, j // self.page], j % self.page]

    def check(self, o, lse, scale=None):
        scale = 1 / np.sqrt(self.D) if scale is None else scale
        o, lse = to64(o), to64(lse)
        terms = self.fp8 and self.T * self.Hq // self.Hkv > 8
        r = 2.0 ** -9 + 2.0 ** -11 if terms else (2.0 ** -11 if self.fp8 else 2.0 ** -8)
        for b in range(self.B):
            n = self.ql[b]
            if n == 0:
                continue
            k, v = self.rows(0, b), self.rows(1, b)
            ref, ref_lse, A, X = paged.tree_attention(to64(self.q[b, :n]), k, v, self.ctx[b],
                                                      None if self.mask is None else self.mask[b], scale)
            dx = (self.D + 16) * 2.0 ** -24 * X
            if terms:
                dx = dx + 2.0 ** -17 * scale * np.abs(to64(self.q[b, :n])).max(-1).T * np.abs(k).sum(-1).max()
            empty = np.isneginf(ref_lse)
            assert np.array_equal(np.isneginf(lse[b, :, :n]), empty)
            gap = np.abs(np.where(empty, 0, lse[b, :, :n]) - np.where(empty, 0, ref_lse))
            assert np.all(gap <= dx + 2.0 ** -18 * (1 + np.where(empty, 0, np.abs(ref_lse)))), (b, gap.max())
            floor = 0.0
            if self.fp8 and self.L[b]:
                j = np.arange(self.L[b])
                s = self.scale[1].cpu().numpy().transpose(0, 2, 1)[self.table[b, j // self.page], j % self.page]
                floor = self.L[b] * 2.0 ** -26 * 448 * float(s.max())
            tol = 2.0 ** -8 * np.abs(ref) + (r + 2 * dx.T[..., None] + 2.0 ** -18) * A + floor
            err = np.abs(o[b, :n] - ref)
            assert np.all(err <= tol), (b, float((err - tol).max()))


def run(p, **more):
    a, kw = p.args()
    o = torch.full((p.B, p.T, p.Hq, p.D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.B, p.Hq, p.T), 6.0, device="cuda")
    ops.attn_decode_paged(*a, out=o, lse=lse, **kw, **more)
    ops.check()
    for b in range(p.B):                               # rows past a sequence's drafts are as they were
        assert torch.all(o[b, p.ql[b]:] == 5.0) and torch.all(lse[b, :, p.ql[b]:] == 6.0)
    return o, lse


SHAPES = [
    # ctx lengths, T, Hq, Hkv, D, page, tree, q_lens
    ([0], 1, 1, 1, 64, 16, False, None),
    ([1, 0, 2], 1, 8, 2, 128, 16, False, None),
    ([15, 16, 17, 127, 128, 129], 1, 4, 1, 128, 16, False, None),
    ([700, 3, 0, 260], 1, 32, 8, 128, 64, False, None),
    ([511], 1, 16, 1, 64, 128, False, None),
    ([90, 1300, 0], 2, 14, 2, 128, 32, False, None),
    ([250, 60, 5], 5, 9, 3, 64, 256, True, None),
    ([120, 0, 127, 1000], 8, 8, 2, 128, 16, True, [8, 6, 0, 7]),
    ([0, 40, 128], 16, 4, 4, 64, 32, True, [16, 1, 15]),
    ([33, 0], 33, 2, 1, 128, 64, True, None),
    ([100, 900], 64, 8, 1, 128, 128, True, [64, 50]),
    ([0, 77], 64, 4, 4, 64, 1024, False, [63, 64]),
    ([2000], 3, 24, 2, 128, 64, True, None),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(str(v) for v in (s[1:6])))
def test_matches_oracle(shape, token_major, fp8):
    ctx, T, Hq, Hkv, D, page, tree, ql = shape
    p = Problem(ctx, T, Hq, Hkv, D, page, fp8, token_major, tree, ql)
    p.check(*run(p))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 6, 40])
def test_many_sequences_share_the_ctas(T, fp8):
    # more units than CTAs, lengths from none to many tiles: units cut at CTA borders everywhere
    rng = np.random.default_rng(T)
    ctx = [int(x) for x in rng.integers(0, 900, 45)]
    ctx[7], ctx[20], ctx[21] = 6000, 0, 0
    p = Problem(ctx, T, 8, 4, 64, 32, fp8, True, T > 1, [int(x) for x in rng.integers(0, T + 1, 45)])
    p.check(*run(p))


@pytest.mark.parametrize("fp8", [False, True])
def test_one_long_sequence_is_cut_over_the_device(fp8):
    p = Problem([40000], 4, 4, 1, 128, 64, fp8, False, True)
    p.check(*run(p))


ROWS = [
    # 9 .. 64 rows (group x drafts), at and next to the tiles of 16, 32 and 64
    ([5, 129, 700], 9, 1, 1, 64, 32, True, [9, 0, 4]),
    ([300, 0, 1], 3, 8, 2, 128, 16, False, None),
    ([1000], 16, 2, 2, 128, 64, True, None),
    ([127, 640], 17, 2, 2, 64, 1024, False, [17, 1]),
    ([2100, 90], 8, 8, 2, 128, 128, True, [8, 8]),
    ([250, 0, 33], 33, 1, 1, 128, 16, True, [33, 2, 20]),
    ([60, 1500], 12, 20, 4, 128, 64, True, None),
    ([100, 0], 64, 2, 2, 64, 64, True, [64, 63]),
    ([64, 128, 65, 191], 64, 1, 1, 128, 32, False, [64, 64, 1, 64]),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("shape", ROWS, ids=lambda s: "x".join(str(v) for v in (s[1:6])))
def test_row_counts_between_the_tiles(shape, token_major, fp8):
    ctx, T, Hq, Hkv, D, page, tree, ql = shape
    p = Problem(ctx, T, Hq, Hkv, D, page, fp8, token_major, tree, ql, case=151)
    p.check(*run(p))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 8, 16, 40])
def test_units_of_many_parts(T, fp8):
    # two sequences over all CTAs, and one with short ones beside it
    for ctx in ([9000, 20000], [30, 25000, 7]):
        p = Problem(ctx, T, 4, 1, 64, 128, fp8, False, True, case=152)
        p.check(*run(p))


@pytest.mark.parametrize("T,Hq", [(1, 4), (4, 4), (8, 4), (16, 4), (40, 4)])
def test_one_key_far_above_many(T, Hq):
    # 40000 keys of probability 2^-19.5 beside one of nearly 1: together they are worth a twentieth
    p = Problem([40000], T, Hq, 1, 64, 1024, fp8=True)
    one = np.float64(np.float32(1 / 448)) * 448
    page, at = int(p.table[0, 0]), 777
    p.q.zero_()
    p.q[..., 0] = 8.0
    for i, (code, sink) in enumerate([(0x00, 0x00), (0xFE, 0x7E)]):
        p.cache[i].fill_(code)
        p.cache[i][page, :, at] = sink
        p.scale[i].fill_(1 / 448)
        p.val[i][:] = 0.0 if i == 0 else -one
    p.cache[0][page, :, at, 0] = 0x7E
    p.scale[0][page, :, at] = 13.5 / 448
    p.val[0][page, :, at, 0] = np.float64(np.float32(13.5 / 448)) * 448
    p.val[1][page, :, at] = one
    p.check(*run(p, scale=0.125), scale=0.125)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 6, 16, 40])
def test_an_infinite_query_element_stays_in_its_row(T, fp8):
    p = Problem([200, 70], T, 4, 1, 64, 32, fp8, tree=True)
    clean = run(p)
    p.q[1, T - 1, 2, 5] = float("inf")
    o, lse = run(p)
    assert torch.isnan(o[1, T - 1, 2]).all()
    o[1, T - 1, 2], lse[1, 2, T - 1] = clean[0][1, T - 1, 2], clean[1][1, 2, T - 1]
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])


def test_logits_far_apart_and_a_given_scale():
    for fp8 in (False, True):
        p = Problem([300, 1500], 3, 8, 2, 128, 16, fp8, tree=True, gain=12.0)
        p.check(*run(p, scale=0.25), scale=0.25)


@pytest.mark.parametrize("T", [1, 8, 36])
@pytest.mark.parametrize("power", [-100, -58, 70, 100])
def test_value_scales_at_the_ends_of_their_range(T, power):
    p = Problem([200, 900, 0], T, 4, 4, 64, 32, fp8=True, tree=T > 1)
    p.scale[1].mul_(2.0 ** power)
    p.val[1] = p.val[1] * 2.0 ** power
    p.check(*run(p))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,Hq", [(6, 4), (20, 8)])
def test_hidden_drafts_may_hold_anything(T, Hq, fp8):
    # draft 1's key and value are NaN or infinite: only rows that see it may show it
    p = Problem([130, 5], T, Hq, 2, 64, 16, fp8, tree=True)
    for b in range(p.B):
        for t in range(T):
            p.mask[b, t] = np.uint64(1 << t) | np.uint64(0b10 if t % 3 == 1 else 0)
    clean = run(p)
    for b in range(p.B):
        j = p.ctx[b] + 1
        pg, at = int(p.table[b, j // p.page]), j % p.page
        for i, bad in ((0, float("nan")), (1, float("inf") if b == 0 else float("nan"))):
            if fp8:
                p.scale[i][pg, :, at] = bad
            else:
                p.cache[i][pg, :, at, 3::7] = bad
    a, kw = p.args()
    o, lse = ops.attn_decode_paged(*a, **kw)
    ops.check()
    sees = [t for t in range(T) if t % 3 == 1]
    blind = [t for t in range(T) if t % 3 != 1]
    assert torch.equal(o[:, blind], clean[0][:, blind]) and torch.equal(lse[:, :, blind], clean[1][:, :, blind])
    assert torch.isnan(lse[:, :, sees]).all() and torch.isnan(o[:, sees]).any(-1).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [4, 40])
def test_a_row_that_sees_nothing(T, fp8):
    p = Problem([0, 50, 0], T, 4, 2, 64, 16, fp8, tree=True)
    p.mask[0, 2] = 0
    p.mask[1, 1] = 0
    p.mask[2, :] = 0
    o, lse = run(p)
    p.check(o, lse)
    assert torch.all(o[0, 2] == 0) and torch.all(o[2] == 0) and torch.isneginf(lse[2]).all()
    assert torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("ctx,ql", [([100, -1], [2, 2]), ([100, 5000], [2, 2]), ([100, 60], [2, 3]), ([100, 60], [-1, 2]),
                                    ([100, 2 ** 31 - 1], [2, 2])])
def test_lengths_out_of_range_write_nothing(ctx, ql):
    p = Problem([100, 60], 2, 4, 2, 64, 16, q_lens=[2, 2])
    a, kw = p.args()
    a = a[:4] + (torch.tensor(ctx, dtype=torch.int32, device="cuda"),)
    kw["q_lens"] = torch.tensor(ql, dtype=torch.int32, device="cuda")
    o = torch.full((2, 2, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 4, 2), 6.0, device="cuda")
    ops.attn_decode_paged(*a, out=o, lse=lse, **kw)
    with pytest.raises(_lib.AttnError, match="length"):
        ops.check()
    assert torch.all(o == 5.0) and torch.all(lse == 6.0)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("page_id", [-1, 10 ** 9, "n_pages"])
def test_a_page_outside_the_cache_is_reported(page_id, T):
    p = Problem([100, 300], T, 4, 2, 64, 16, fp8=True)
    good = run(p)
    p.table[1, 3] = p.n_pages if page_id == "n_pages" else page_id
    a, kw = p.args()
    o, lse = ops.attn_decode_paged(*a, **kw)
    with pytest.raises(_lib.AttnError, match="page number"):
        ops.check()
    assert torch.equal(o[0], good[0][0]) and torch.equal(lse[0], good[1][0])     # the other sequence stands


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 40])
def test_graph_replays_read_the_lengths_they_find(T, fp8):
    p = Problem([900, 1200, 17], T, 8, 2, 128, 32, fp8, tree=T > 1)
    a, kw = p.args()
    B, Hq, D = p.B, p.Hq, p.D
    ws = torch.empty(ops.decode_paged_workspace_bytes(B, T, Hq, 2, D, 32, p.max_pages), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(a[0]), torch.empty((B, Hq, T), device="cuda")
    ops.attn_decode_paged(*a, out=o, lse=lse, workspace=ws, **kw)              # first call: loads the kernels
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.attn_decode_paged(*a, out=o, lse=lse, workspace=ws, **kw)
    for ctx in ([900, 1200, 17], [10, 1200, 0], [900, 0, 3]):
        a[4].copy_(torch.tensor(ctx, dtype=torch.int32))
        want = ops.attn_decode_paged(*a, **kw)
        ws.fill_(0xFF)                                                        # the workspace carries nothing over
        g.replay()
        ops.check()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_same_bits_from_run_to_run_and_on_another_stream():
    for T, fp8 in ((1, True), (8, False), (40, True), (40, False)):
        p = Problem([3000, 700, 64], T, 8, 2, 128, 64, fp8, tree=T > 1)
        a, kw = p.args()
        first = ops.attn_decode_paged(*a, **kw)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        outs = [ops.attn_decode_paged(*a, stream=st if i % 2 else None, **kw) for i in range(20)]
        torch.cuda.current_stream().wait_stream(st)
        ops.check()
        for o, lse in outs:
            assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_contiguous_decoding_agrees():
    # a cache [B, S, Hkv, D] is B * S / page token-major pages
    B, S, Hq, Hkv, D, page = 3, 768, 16, 4, 128, 64
    q, k, v = (torch.from_numpy(synth.normal(s, synth.seed_for(151, i))).to(torch.bfloat16).cuda()
               for i, s in enumerate([(B, 1, Hq, D), (B, S, Hkv, D), (B, S, Hkv, D)]))
    table = torch.arange(B * S // page, dtype=torch.int32, device="cuda").view(B, -1)
    ctx = torch.full((B,), S - 1, dtype=torch.int32, device="cuda")
    o, lse = ops.attn_decode_paged(q, k.view(-1, page, Hkv, D), v.view(-1, page, Hkv, D), table, ctx, token_major=True)
    o2, lse2 = ops.attn_decode(q, k, v)
    ops.check()
    # both round numerators to bf16 (2^-8 of sum p |v| <= max |v|, about 5) and the output
    assert (o.float() - o2.float()).abs().max() <= 2 * 2.0 ** -8 * 5 * 0.3
    assert (lse - lse2).abs().max() <= 1e-4


def test_offsets_beyond_32_bits():
    # the only used pages lie past 2^32 elements of a bf16 cache
    Hkv, page, D = 8, 1024, 128
    n_pages = 2 ** 32 // (Hkv * page * D) + 3
    if torch.cuda.mem_get_info()[0] < 3 * n_pages * Hkv * page * D * 2:
        pytest.skip("not enough device memory")
    kc, vc = (torch.empty((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = (torch.from_numpy(synth.normal(s, synth.seed_for(152, i))).to(torch.bfloat16).cuda()
               for i, s in enumerate([(1, 2, 16, D), (1030, Hkv, D), (1030, Hkv, D)]))
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    j = torch.arange(1030, device="cuda")
    ops.kv_cache_append(k, v, kc, vc, table[0].long()[j // page] * page + j % page)
    ctx = torch.tensor([1028], dtype=torch.int32, device="cuda")
    far = ops.attn_decode_paged(q, kc, vc, table, ctx)
    near_k, near_v = kc[-2:].flip(0).contiguous(), vc[-2:].flip(0).contiguous()
    near = ops.attn_decode_paged(q, near_k, near_v, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), ctx)
    ops.check()
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_then_drafts_then_read_back(fp8):
    """A serving run: a prompt's keys and values are rotated and written, a tree of drafts follows and
    attends, the accepted path is written again behind the prompt, one token decodes, and the
    sequence is read back and attended whole."""
    Hq, Hkv, D, page, n, T = 4, 4, 64, 16, 150, 6
    qkv = torch.from_numpy(synth.normal((n + T + 1, Hq + 2 * Hkv, D), synth.seed_for(153, 0))).to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cs = ops.rope_scaled_table(256, D, scaling="linear", factor=2.0)
    dt, sc = (torch.uint8, 2) if fp8 else (torch.bfloat16, 0)
    kc, vc = (torch.zeros((12, Hkv, page, D), dtype=dt, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((12, Hkv, page), device="cuda") for _ in range(2)) if sc else (None, None)
    table = torch.randperm(12, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()[None]

    def write(tokens, places, depth):
        places, depth = torch.tensor(places, device="cuda"), torch.tensor(depth, dtype=torch.int32, device="cuda")
        slots = table[0].long()[places // page] * page + places % page
        return ops.rope_kv_cache_append(q[tokens], k[tokens], v[tokens], cs, depth, kc, vc, slots, ks, vs)

    write(list(range(n)), list(range(n)), list(range(n)))
    parent = [-1, 0, 0, 1, 2, 4]
    depth, mask = [], []
    for t, up in enumerate(parent):
        depth.append(n + (0 if up < 0 else depth[up] - n + 1))
        mask.append((1 << t) | (mask[up] if up >= 0 else 0))
    drafts = list(range(n, n + T))
    tq = write(drafts, drafts, depth)
    ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
    tree, _ = ops.attn_decode_paged(tq[None], kc, vc, table, ctx, ks, vs,
                                    tree_mask=torch.tensor([mask], device="cuda"))
    path = [0, 2, 4, 5]                                 # accepted: written again, in line
    write([n + i for i in path], list(range(n, n + 4)), list(range(n, n + 4)))
    last = write([n + T], [n + 4], [n + 4])
    one, one_lse = ops.attn_decode_paged(last[None], kc, vc, table, ctx + 4, ks, vs)
    total = n + 5
    ko, vo = ops.kv_cache_gather(kc, vc, table, torch.tensor([0, total], dtype=torch.int32, device="cuda"), total, ks, vs)
    whole_q = ops.rope_apply(torch.cat([q[:n], q[[n + i for i in path]], q[[n + T]]]), cs)
    cu = torch.tensor([0, total], dtype=torch.int32, device="cuda")
    o, lse = ops.attn_fwd_varlen(whole_q, ko, vo, cu, total, causal=True)
    ops.check()
    # read-back rounds code * scale to bf16 (2^-8 of each k and v), numerators and outputs round too:
    # logits move by 2^-8 scale sum |q k| <= 2^-8 * 8 * 3, outputs by that and three roundings of |v| <= 5
    tol = (2.0 ** -8 * 24 * 0.25 + 3 * 2.0 ** -8) * 2
    assert (o[-1].float() - one[0, 0].float()).abs().max() <= tol
    assert (lse[:, -1] - one_lse[0, :, 0]).abs().max() <= 2.0 ** -8 * 24
    for i, t in enumerate(path):                        # the tree's rows on the accepted path
        assert (o[n + i].float() - tree[0, t].float()).abs().max() <= tol


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 36])
def test_each_launch_sees_the_one_before(T, fp8):
    # the launches may overlap at their ends, so: every step writes new rows over the old ones and attends to
    # them at once, with new lengths, without a synchronisation between; every result must be the one
    # that the same inputs give by themselves
    B, Hq, Hkv, D, page, n = 5, 4, 2, 64, 16, 333
    qkv = torch.from_numpy(synth.normal((6, B * n, Hq + 2 * Hkv, D), synth.seed_for(154, 0))).to(torch.bfloat16).cuda()
    dt = torch.uint8 if fp8 else torch.bfloat16
    table = torch.randperm(B * 25, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda().view(B, 25)
    j = torch.arange(n, device="cuda")
    slots = (table.long()[:, j // page] * page + j % page).reshape(-1)
    pos = j.to(torch.int32).repeat(B)
    cs = ops.rope_scaled_table(512, D)
    step_lens = [torch.tensor([n - T - 7 * (i + b) for b in range(B)], dtype=torch.int32, device="cuda") for i in range(6)]

    def new():
        kc, vc = (torch.zeros((B * 25, Hkv, page, D), dtype=dt, device="cuda") for _ in range(2))
        sc = [torch.ones((B * 25, Hkv, page), device="cuda") for _ in range(2)] if fp8 else [None, None]
        return kc, vc, sc

    def step(i, kc, vc, sc, ctx):
        x = qkv[i]
        q = ops.rope_kv_cache_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cs, pos, kc, vc, slots, *sc)
        return ops.attn_decode_paged(q.view(B, n, Hq, D)[:, n - T:].contiguous(), kc, vc, table, ctx, *sc)

    kc, vc, sc = new()
    ctx = torch.empty(B, dtype=torch.int32, device="cuda")
    got = []
    for rep in range(3):
        for i in range(6):
            ctx.copy_(step_lens[i])
            got.append(step(i, kc, vc, sc, ctx))
    ops.check()
    for i in range(6):
        kc, vc, sc = new()
        torch.cuda.synchronize()
        want = step(i, kc, vc, sc, step_lens[i])
        ops.check()
        for rep in range(3):
            assert torch.equal(got[6 * rep + i][0], want[0]) and torch.equal(got[6 * rep + i][1], want[1]), (rep, i)


KINDS = [(1, 8, 2, False), (4, 8, 2, False), (8, 8, 2, False), (16, 8, 2, False), (40, 8, 2, False), (1, 8, 2, True), (3, 8, 2, True),
         (8, 8, 2, True), (16, 8, 2, True), (40, 8, 2, True)]      # T, Hq, Hkv, fp8: each kernel and row tile


@pytest.mark.parametrize("T,Hq,Hkv,fp8", KINDS)
def test_calls_on_two_streams_at_once(T, Hq, Hkv, fp8):
    p = [Problem(c, T, Hq, Hkv, 128, 64, fp8, tree=True, case=155 + i) for i, c in enumerate([[2000, 90, 700], [30, 5000]])]
    args = [x.args() for x in p]
    want = [ops.attn_decode_paged(*a, **kw) for a, kw in args]
    ops.check()
    need = [ops.decode_paged_workspace_bytes(x.B, T, Hq, Hkv, 128, 64, x.max_pages) for x in p]
    streams = [torch.cuda.Stream() for _ in p]
    for i, x in enumerate(p):
        streams[i].wait_stream(torch.cuda.current_stream())
    got = [[], []]
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in need]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (a, kw) in enumerate(args):
            got[i].append(ops.attn_decode_paged(*a, workspace=ws[i], stream=streams[i], **kw))
    torch.cuda.synchronize()
    ops.check()
    for w, outs in zip(want, got):
        for o, lse in outs:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("T,Hq,Hkv,fp8", KINDS)
def test_the_workspace_is_not_left(T, Hq, Hkv, fp8):
    p = Problem([9000, 40, 1300], T, Hq, Hkv, 64, 32, fp8, tree=True)
    need = ops.decode_paged_workspace_bytes(p.B, T, Hq, Hkv, 64, 32, p.max_pages)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    p.check(*run(p, workspace=ws[:need]))
    assert torch.all(ws[need:] == 0xA5)
    with pytest.raises(_lib.AttnError):
        run(p, workspace=ws[:need - 16])


@pytest.mark.parametrize("T,Hq,Hkv,fp8", KINDS)
def test_two_graphs_share_a_workspace(T, Hq, Hkv, fp8):
    p = [Problem(c, T, Hq, Hkv, 128, 128, fp8, tree=True, case=157 + i) for i, c in enumerate([[4000, 90], [130, 2500]])]
    args = [x.args() for x in p]
    want = [ops.attn_decode_paged(*a, **kw) for a, kw in args]
    ops.check()
    ws = torch.empty(max(ops.decode_paged_workspace_bytes(x.B, T, Hq, Hkv, 128, 128, x.max_pages) for x in p),
                     dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for a, kw in args:
        o = torch.empty_like(want[len(outs)][0]), torch.empty_like(want[len(outs)][1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.attn_decode_paged(*a, workspace=ws, out=o[0], lse=o[1], **kw)
        graphs.append(g)
        outs.append(o)
    for _ in range(5):
        for o in outs:
            o[0].zero_()
            o[1].zero_()
        for g in graphs:
            g.replay()
        ops.check()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


@pytest.mark.parametrize("T,Hq,Hkv,fp8", KINDS)
def test_what_lies_outside_is_refused_by_every_kernel(T, Hq, Hkv, fp8):
    # a page outside the cache is reported and not read; lengths out of range write nothing
    p = Problem([700, 90], T, Hq, Hkv, 64, 64, fp8, tree=True)
    clean = run(p)
    good = p.table.copy()
    p.table[0, 3] = p.n_pages
    a, kw = p.args()
    o = torch.full_like(clean[0], 5.0)
    lse = torch.full_like(clean[1], 6.0)
    ops.attn_decode_paged(*a, out=o, lse=lse, **kw)
    with pytest.raises(_lib.AttnError, match="page"):
        ops.check()
    assert torch.equal(o[1], clean[0][1]) and torch.equal(lse[1], clean[1][1])
    p.table[:] = good
    p.ctx[0] = p.max_pages * p.page + 1
    a, kw = p.args()
    o.fill_(5.0)
    lse.fill_(6.0)
    ops.attn_decode_paged(*a, out=o, lse=lse, **kw)
    with pytest.raises(_lib.AttnError):
        ops.check()
    assert torch.all(o == 5.0) and torch.all(lse == 6.0)
    p.ctx[0] = 700
    again = run(p)
    assert torch.equal(again[0], clean[0]) and torch.equal(again[1], clean[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 5, 20, 33])
def test_a_thousand_sequences(T, fp8):
    rng = np.random.default_rng(159)
    ctx = rng.integers(0, 200, 1024).tolist()
    ql = rng.integers(0, T + 1, 1024).tolist()
    p = Problem(ctx, T, 3, 1, 64, 128, fp8, False, True, ql, case=160)
    p.check(*run(p))


@pytest.mark.parametrize("T,Hq,Hkv,fp8", KINDS)
def test_no_drafts_at_all(T, Hq, Hkv, fp8):
    # nothing is written, and the call after it is none the worse
    p = Problem([700, 90, 0], T, Hq, Hkv, 64, 64, fp8, tree=True, q_lens=[0, 0, 0])
    o, lse = run(p)
    assert torch.all(o == 5.0) and torch.all(lse == 6.0)
    p = Problem([700, 90, 0], T, Hq, Hkv, 64, 64, fp8, tree=True, q_lens=[0, T, 0])
    p.check(*run(p))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 7, 30])
def test_a_zero_value_scale_gives_zeros(T, fp8):
    p = Problem([300, 20], T, 2, 1, 64, 32, fp8, tree=True)
    if fp8:
        p.scale[1].zero_()
    else:
        p.cache[1].zero_()
    o, lse = run(p)
    assert torch.all(o == 0) and torch.isfinite(lse).all()
