"""The paged K/V cache, chunk attention over it and cross attention on the GPU against the fp64 oracle.

Tolerances (u = half a step: 2^-8 bf16, 2^-11 f16, 2^-24 fp32; A = softmax-weighted mean of |v|):
the output's rounding 2^-8 |o|; the roundings before the second product:
 - INT8 values, f16: a weight, a scale and a value times its scale are rounded once each, 3 2^-11 A. What is below
   2^-14 loses up to 2^-25 instead: a weight that of the largest value, n 2^-24 max|v| for n of them; a value, which
   enters as code * (s c) / 4096 with s c >= 1 for the largest scale s, 2^-25 4096 s <= 2^-13 max|v| / 127 < 2^-19 max|v|,
   times weights that sum to 1. (Values enter as code * (s c) with s c >= 2^5 for the largest scale, which loses less.)
 - bf16 values: a weight p enters as p (1 + e), |e| <= 2^-8, and the sum that divides as it entered, so that o moves by
   sum p e (v - o) / sum p (1 + e), at most 2^-8 (A + |o|) (1 + 2^-7).
A logit x of d products in fp32 is off by dx = (d + 4) 2^-24 scale sum|q||k|, which moves a weight by
the factor 1 +- 2 dx and so o by 2 dx 2 A; the exponential and the fp32 sums over n keys add (n + 8) 2^-22 A.
lse: dx + (n + 8) 2^-22 + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _bf16(rng, shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * scale).to(torch.bfloat16)


class Setup:
    """Ragged sequences in a shuffled page pool. ``past`` tokens are placed by the test (oracle codes), the new
    ones by ``write``. Pages and rows no token has hold poison."""

    def __init__(self, bsva, lens, H, d, page, dtype, seed=0, tail=0, lead=0, poison=True, mag=1.0):
        rng = np.random.default_rng(seed)
        self.bsva, self.lens, self.H, self.d, self.page, self.dtype = bsva, lens, H, d, page, dtype
        S = len(lens)
        per = max(1, max(-(-kv // page) for _, kv in lens))
        n_pages = sum(-(-kv // page) for _, kv in lens) + 2
        order = np.random.default_rng(seed + 1).permutation(n_pages)   # apart from the tokens, which no page size changes
        self.table = np.full((S, per), -7, np.int32)
        at = 0
        for s, (_, kv) in enumerate(lens):
            n = -(-kv // page)
            self.table[s, :n] = order[at:at + n]
            at += n
        self.kv = [[(_bf16(rng, (kv, H, d)) * torch.from_numpy(np.exp(rng.standard_normal((kv, H, 1)) * mag)
                                                                .astype(np.float32)).to(torch.bfloat16))
                    for _, kv in lens] for _ in range(2)]
        starts = [lead]
        for n, _ in lens:
            starts.append(starts[-1] + n)
        self.starts, self.T = starts, starts[-1] + tail
        new = [torch.zeros((self.T, H, d), dtype=torch.bfloat16) for _ in range(2)]
        for z in range(2):
            for s, (n, kv) in enumerate(lens):
                if n and kv >= n:
                    new[z][starts[s]:starts[s + 1]] = self.kv[z][s][kv - n:]
        self.new = [x.cuda() for x in new]
        # the pool: poison everywhere, then the past
        shape = (n_pages, H, page, d)
        if dtype == torch.int8:
            pool = [rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2)]
            scale = [np.full(shape[:3], NAN if poison else 1.0, np.float32) for _ in range(2)]
        else:
            pool = [np.full(shape, NAN if poison else 1.0, np.float32) for _ in range(2)]
        self.values = [[None] * S for _ in range(2)]    # what the cache stands for, [kv, H, d] fp64
        for z in range(2):
            for s, (n, kv) in enumerate(lens):
                x = self.kv[z][s].float().numpy()
                codes, sc = paged.quantize_rows(x)
                self.values[z][s] = paged.dequantize_rows(codes, sc) if dtype == torch.int8 else x.astype(np.float64)
                t = np.arange(max(kv - n, 0))
                pg = self.table[s][t // page]
                if dtype == torch.int8:
                    pool[z][pg, :, t % page] = codes[t]
                    scale[z][pg, :, t % page] = sc[t]
                else:
                    pool[z][pg, :, t % page] = x[t]
        if dtype == torch.int8:
            self.cache = bsva.PagedKVCache.over(*[torch.from_numpy(x).cuda() for x in pool],
                                                *[torch.from_numpy(x).cuda() for x in scale])
        else:
            self.cache = bsva.PagedKVCache.over(*[torch.from_numpy(x).to(torch.bfloat16).cuda() for x in pool])
        i32 = dict(dtype=torch.int32, device="cuda")
        self.batch = bsva.PagedBatch(torch.tensor(starts, **i32), torch.tensor([kv for _, kv in lens], **i32),
                                     torch.from_numpy(self.table).cuda(), max(1, max(n for n, _ in lens)),
                                     max(1, max(kv for _, kv in lens)))
        self.rng = rng

    def queries(self, Hq, scale=1.0):
        return _bf16(self.rng, (self.T, Hq, self.d), scale)

    def check(self, q, out, lse, causal=True, window=0, scale=None):
        Hq = q.shape[1]
        G = Hq // self.H
        o_, l_ = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for s, (n, kv) in enumerate(self.lens):
            ok = paged.visible(n, kv, causal, window)
            rows = slice(self.starts[s], self.starts[s] + n)
            for h in range(Hq):
                close(q[rows, h].double().numpy(), self.values[0][s][:, h // G], self.values[1][s][:, h // G], ok,
                      o_[rows, h], l_[rows, h], scale, self.dtype, f"sequence {s} head {h}")


def close(q, k, v, ok, o, lse, scale, dtype, where):
    """Compares one head's rows with the oracle within the derived bounds."""
    n, d = q.shape
    if n == 0:
        return
    sc = 1 / math.sqrt(d) if scale is None else scale
    ro, rl, A = paged.attention_rows(q, k, v, ok, sc)
    keys = max(1, ok.shape[1])
    dx = ((d + 4) * 2.0 ** -24 * sc * np.where(ok, np.abs(q) @ np.abs(k).T, 0).max(1, initial=0))[:, None]
    vmax = np.abs(np.where(ok.any(0)[:, None], v, 0)).max(initial=0)
    u = 3 * 2.0 ** -11 if dtype == torch.int8 else 2.0 ** -8
    tol = 2.0 ** -8 * np.abs(ro) + (u + 4 * dx + (keys + 8) * 2.0 ** -22) * A * 1.01 + 1e-38
    if dtype == torch.int8:
        tol += (keys * 2.0 ** -24 + 2.0 ** -19) * vmax
    else:
        tol += 2.0 ** -8 * np.abs(ro)
    bad = ~(np.abs(o - ro) <= tol)
    assert not bad.any(), f"{where}: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(o - ro) / tol)} of the bound"
    dead = ~np.isfinite(rl)
    assert (lse[dead] == -np.inf).all() and (o[dead] == 0).all(), where
    tl = dx[:, 0] + (keys + 8) * 2.0 ** -22 + 2.0 ** -22 * np.abs(np.where(dead, 0, rl))
    assert (np.abs(np.where(dead, 0, lse) - np.where(dead, 0, rl)) <= np.where(dead, 1, tl)).all(), where


def _attend(st, Hq, causal=True, window=0, scale=None, qscale=1.0, write=True):
    if write:
        st.cache.write(st.new[0], st.new[1], st.batch)
    q = st.queries(Hq, qscale)
    ws = st.cache.new_workspace(st.batch, Hq, st.T)
    out = torch.full((st.T, Hq, st.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((st.T, Hq), 7.0, device="cuda")
    st.cache.attend(q.cuda(), st.batch, causal=causal, window=window, softmax_scale=scale or 0.0, with_lse=True, out=out,
                    lse=lse, workspace=ws)
    st.bsva.check_status(ws)
    for x in (out, lse):       # rows before the first and behind the last sequence
        assert (x[:st.starts[0]] == 7).all() and (x[st.starts[-1]:] == 7).all()
    st.check(q, out, lse, causal, window, scale)
    return q, out, lse, ws


RAGGED = [(5, 5), (0, 17), (1, 130), (33, 100), (16, 16)]


# ---------------------------------------------------------------------------------------- write and read
@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("d,page,H", [(128, 16, 3), (64, 32, 1), (64, 256, 2), (128, 128, 5)])
def test_write_then_read(gpu_lib, dtype, d, page, H):
    st = Setup(gpu_lib, RAGGED, H, d, page, dtype, seed=d + page, tail=3, lead=2)
    before = [x.clone() for x in (st.cache.k, st.cache.v)]
    ws = st.cache.new_workspace(st.batch, H, st.T)
    fused = torch.cat([st.new[0], st.new[1], st.new[0]], 1)      # a fused projection: k and v are slices of its rows
    st.cache.write(fused[:, :H], fused[:, H:2 * H], st.batch, workspace=ws)
    gpu_lib.check_status(ws)
    for z, pool in enumerate((st.cache.k, st.cache.v)):
        mine = torch.zeros(pool.shape[0], pool.shape[2], dtype=torch.bool)
        for s, (n, kv) in enumerate(st.lens):
            t = np.arange(kv)
            pg, off = st.table[s][t // page], t % page
            got = pool.cpu().float().numpy()[pg, :, off]
            x = st.kv[z][s].float().numpy()
            if dtype == torch.int8:
                codes, sc = paged.quantize_rows(x)
                assert np.array_equal(got, codes.astype(np.float32))
                assert np.array_equal((st.cache.k_scale, st.cache.v_scale)[z].cpu().numpy()[pg, :, off], sc)
            else:
                assert np.array_equal(got, x)
            mine[pg, off] = True
        keep = ~mine[:, None, :, None].expand(pool.shape)
        a, b = pool.cpu()[keep], before[z].cpu()[keep]           # rows without a token are as they were
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
    for first in (None, [0, 20, 7, 99, 3]):
        ft = None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda")
        L = 133 if first is None else 140
        outs = st.cache.read(st.batch, first=ft, length=L, workspace=ws)
        gpu_lib.check_status(ws)
        for z in range(2):
            got = outs[z].cpu()
            assert got.shape == (len(RAGGED), H, L, d)
            for s, (_, kv) in enumerate(st.lens):
                f = 0 if first is None else min(first[s], kv)
                want = torch.from_numpy(st.values[z][s][f:].astype(np.float32)).to(torch.bfloat16).transpose(0, 1)
                assert torch.equal(got[s, :, :kv - f], want)
                assert (got[s, :, kv - f:] == 0).all()


def test_write_zero_subnormal_and_tie_rows(gpu_lib):
    st = Setup(gpu_lib, [(40, 40)], 2, 64, 16, torch.int8, seed=3)
    x = st.new[0]
    x[0] = 0
    x[1] = 1e-39
    x[2, :, ::2] = -3e-38
    x[3] *= 2.0 ** 100
    x[4] = (torch.arange(64, device="cuda") - 31.5).to(torch.bfloat16) * 2 + 0.0   # halves of a code against amax 127
    x[4, :, 0] = 127
    st.cache.write(x, x, st.batch)
    codes, sc = paged.quantize_rows(x.float().cpu().numpy())
    t = np.arange(40)
    pg = st.table[0][t // 16]
    assert np.array_equal(st.cache.k.cpu().numpy()[pg, :, t % 16], codes)
    assert np.array_equal(st.cache.v_scale.cpu().numpy()[pg, :, t % 16], sc)


# ---------------------------------------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,H", [(1, 3), (5, 2), (8, 1), (3, 1)])
def test_single_tokens(gpu_lib, dtype, d, G, H):
    lens = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 63), (1, 65), (1, 700), (0, 9), (1, 1003)]
    _attend(Setup(gpu_lib, lens, H, d, 16, dtype, seed=G), G * H)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("d,page,G,H", [(64, 16, 1, 2), (128, 32, 2, 1), (128, 64, 7, 1), (64, 128, 4, 2), (128, 256, 1, 1)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 40), (True, 100000), (False, 0)])
def test_chunks(gpu_lib, dtype, d, page, G, H, causal, window):
    lens = [(5, 5), (0, 17), (1, 130), (33, 100), (16, 16), (129, 400), (2, 900), (64, 128)]
    _attend(Setup(gpu_lib, lens, H, d, page, dtype, seed=page + G, tail=2, lead=1), G * H, causal, window)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("n,kv,G,H,d,window", [(300, 2000, 1, 2, 128, 0), (257, 257, 1, 1, 64, 0), (256, 1280, 3, 1, 128, 0),
                                               (700, 1500, 1, 1, 128, 333), (127, 5000, 2, 1, 64, 0)])
def test_longer_chunks(gpu_lib, dtype, n, kv, G, H, d, window):
    _attend(Setup(gpu_lib, [(n, kv)], H, d, 64, dtype, seed=n), G * H, True, window)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("n,page", [(1, 16), (1, 64), (150, 16), (150, 128), (150, 256)])
def test_tokens_before_the_window_are_gone(gpu_lib, dtype, n, page):
    window, lens = 70, [(n, 777), (n, 300)]
    st = Setup(gpu_lib, lens, 2, 64, page, dtype, seed=n + page)
    table = st.table.copy()
    for s, (_, kv) in enumerate(lens):
        first = kv - n - window + 1            # the first token that some row sees
        for pool, scale in ((st.cache.k, st.cache.k_scale), (st.cache.v, st.cache.v_scale)):
            t = np.arange(first // page * page, first)
            if dtype == torch.int8:
                scale[st.table[s][t // page], :, t % page] = NAN
            else:
                pool[st.table[s][t // page], :, t % page] = NAN
        table[s, :first // page] = -1
    st.batch.page_table.copy_(torch.from_numpy(table))
    _attend(st, 4, True, window)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 200])
def test_rows_without_keys(gpu_lib, dtype, n):
    # sequences shorter than their chunk: the first rows see nothing; a sequence without any key
    st = Setup(gpu_lib, [(n, n), (n, 0), (n, n // 3), (1, 0)], 2, 64, 16, dtype, seed=n)
    st.cache.write(st.new[0], st.new[1], st.batch)      # the short ones' first tokens have no place and are reported
    for s, (m, kv) in enumerate(st.lens):               # ... their keys are placed here
        for z, pool in enumerate((st.cache.k, st.cache.v)):
            for t in range(kv):
                x = st.kv[z][s][t].float().numpy()
                if dtype == torch.int8:
                    c, sc = paged.quantize_rows(x)
                    pool[st.table[s][t // 16], :, t % 16] = torch.from_numpy(c).cuda()
                    (st.cache.k_scale, st.cache.v_scale)[z][st.table[s][t // 16], :, t % 16] = torch.from_numpy(sc).cuda()
                else:
                    pool[st.table[s][t // 16], :, t % 16] = torch.from_numpy(x).to(torch.bfloat16).cuda()
    _attend(st, 4, write=False)
    _attend(st, 4, causal=False, write=False)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("qscale,mag", [(0.0, 1.0), (30.0, 1.0), (1.0, 6.0), (8.0, 3.0)])
def test_large_logits_and_scales_of_many_sizes(gpu_lib, dtype, n, qscale, mag):
    # equal weights; near one-hot weights; tokens whose sizes (and so scales) differ by e^12 and more
    _attend(Setup(gpu_lib, [(n, 600), (n, 90)], 2, 128, 32, dtype, seed=n, mag=mag), 2, qscale=qscale)


@pytest.mark.parametrize("n", [1, 40])
def test_zero_rows_and_softmax_scale(gpu_lib, n):
    st = Setup(gpu_lib, [(n, 300)], 1, 64, 16, torch.int8, seed=9)
    st.cache.write(st.new[0], st.new[1], st.batch)
    st.cache.v_scale.zero_()           # every value row is zero: scale 0
    q, out, lse, _ = st.queries(2), None, None, None
    out, lse = st.cache.attend(q.cuda(), st.batch, softmax_scale=0.3, with_lse=True)
    assert (out == 0).all()
    st.values[1][0][:] = 0
    st.check(q, out, lse, scale=0.3)


def test_page_sizes_agree_and_runs_repeat(gpu_lib):
    # the same tokens in pages of other sizes: the keys meet in the same order, so the bits agree; and twice
    for n in (1, 200):
        first = None
        for page in (16, 64, 256):
            st = Setup(gpu_lib, [(n, 500), (min(n, 77), 77)], 2, 128, page, torch.int8, seed=4)
            st.cache.write(st.new[0], st.new[1], st.batch)
            q = _bf16(np.random.default_rng(1), (st.T, 4, 128)).cuda()
            a, la = st.cache.attend(q, st.batch, with_lse=True)
            b, lb = st.cache.attend(q, st.batch, with_lse=True)
            assert torch.equal(a, b) and torch.equal(la, lb)
            first = (a, la) if first is None else first
            assert torch.equal(a, first[0]) and torch.equal(la, first[1])


def test_generation_step_by_step(gpu_lib):
    """Prompt, then tokens one at a time, against the whole sequence in one chunk; and the cache read back enters
    cross attention as keys."""
    H, G, d, page, n = 2, 3, 64, 16, 50
    st = Setup(gpu_lib, [(n, n), (n, n)], H, d, page, torch.int8, seed=11)
    q, out, lse, _ = _attend(st, G * H)
    k, v = st.cache.read(st.batch)
    one = gpu_lib.PagedKVCache(st.cache.n_pages, page, H, d)
    i32 = dict(dtype=torch.int32, device="cuda")
    steps = [(0, 30)] + [(t, t + 1) for t in range(30, n)]
    for a, b in steps:
        m = b - a
        batch = gpu_lib.PagedBatch(torch.tensor([0, m, 2 * m], **i32), torch.tensor([b, b], **i32), st.batch.page_table, m, b)
        rows = torch.cat([torch.arange(a, b), torch.arange(n + a, n + b)])
        ws = one.new_workspace(batch, G * H)
        one.write(st.new[0][rows], st.new[1][rows], batch, workspace=ws)
        o, ls = one.attend(q.cuda()[rows], batch, with_lse=True, workspace=ws)
        gpu_lib.check_status(ws)
        # two results of the same rows, each within the bounds of check(): compare both with the oracle
        out[rows], lse[rows] = o, ls
    st.check(q, out, lse)
    k1, v1 = one.read(st.batch)
    assert torch.equal(k1, k) and torch.equal(v1, v)
    x = _bf16(np.random.default_rng(5), (2, 2, 9, d)).cuda()
    o, ls = gpu_lib.cross_attn_fwd(x, k, v, with_lse=True)
    for b in range(2):
        for h in range(2):
            close(x[b, h].double().cpu().numpy(), k[b, h].double().cpu().numpy(), v[b, h].double().cpu().numpy(),
                  np.ones((9, n), bool), o[b, h].double().cpu().numpy(), ls[b, h].double().cpu().numpy(), None,
                  torch.bfloat16, f"batch {b} head {h}")


def test_prefix_pages_shared_by_sequences(gpu_lib):
    st = Setup(gpu_lib, [(4, 100), (4, 100)], 2, 128, 32, torch.int8, seed=21)
    table = st.table.copy()
    table[1, :2] = table[0, :2]        # 64 tokens of prefix in common
    st.batch.page_table.copy_(torch.from_numpy(table))
    for z in range(2):
        st.values[z][1][:64] = st.values[z][0][:64]
    _attend(st, 6)


def test_graph_replays_with_other_lengths_and_streams(gpu_lib):
    H, G, d = 2, 4, 128
    big = Setup(gpu_lib, [(1, 900), (1, 40), (1, 333)], H, d, 16, torch.int8, seed=31)
    ws = big.cache.new_workspace(big.batch, G * H)
    q = big.queries(G * H)
    qd = q.cuda()
    out, lse = torch.zeros_like(qd), torch.zeros((big.T, G * H), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        big.cache.write(big.new[0], big.new[1], big.batch, workspace=ws)
        big.cache.attend(qd, big.batch, with_lse=True, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        big.cache.write(big.new[0], big.new[1], big.batch, workspace=ws)
        big.cache.attend(qd, big.batch, with_lse=True, out=out, lse=lse, workspace=ws)
    out.zero_()
    graph.replay()
    gpu_lib.check_status(ws)
    big.check(q, out, lse)
    # shorter sequences through the same graph: the tokens now cached last are attended from the new ends
    lens = [(1, 17), (1, 40), (0, 200)]
    big.batch.kv_len.copy_(torch.tensor([kv for _, kv in lens], dtype=torch.int32))
    big.batch.q_start.copy_(torch.tensor([0, 1, 2, 2], dtype=torch.int32))
    graph.replay()
    gpu_lib.check_status(ws)
    for z in range(2):                 # token 16 of sequence 0 was written anew
        big.values[z][0][16] = big.values[z][0][899]
        big.values[z][0] = big.values[z][0][:17]
        big.values[z][2] = big.values[z][2][:200]
    big.lens = lens
    big.check(q, out, lse)


# -------------------------------------------------------------------- device arrays that break their bounds
def test_broken_bounds_are_reported_and_neighbours_are_right(gpu_lib):
    H, d = 2, 64
    for n in (1, 40):
        st = Setup(gpu_lib, [(n, 120), (n, 64)], H, d, 16, torch.int8, seed=41, poison=False)
        q, out, lse, ws = _attend(st, 4)
        good = st.batch.page_table.clone()
        for bad in (st.cache.n_pages, -1, 2 ** 31 - 1, -2 ** 31):
            st.batch.page_table[0, 1] = bad
            o, ls = st.cache.attend(q.cuda(), st.batch, with_lse=True, workspace=ws)
            with pytest.raises(gpu_lib.BsvaError) as e:
                gpu_lib.check_status(ws)
            assert e.value.code == 6
            assert torch.equal(o[n:], out[n:]) and torch.equal(ls[n:], lse[n:])
            st.cache.read(st.batch, workspace=ws)
            with pytest.raises(gpu_lib.BsvaError):
                gpu_lib.check_status(ws)
        st.batch.page_table.copy_(good)
        st.batch.page_table[1, (64 - n) // 16] = st.cache.n_pages
        before = st.cache.k.clone()
        st.cache.write(st.new[0], st.new[1], st.batch, workspace=ws)
        with pytest.raises(gpu_lib.BsvaError):
            gpu_lib.check_status(ws)
        assert torch.equal(before, st.cache.k)      # the others rewrote what they had, the bad one nothing
        st.batch.page_table.copy_(good)
        for name, bad in (("kv_len", [200, 64]), ("kv_len", [-3, 64]), ("q_start", [0, n, 2 * n + 9]),
                          ("q_start", [5, 0, 2]), ("q_start", [-1, n, 2 * n])):
            t = getattr(st.batch, name)
            keep = t.clone()
            t.copy_(torch.tensor(bad, dtype=torch.int32))
            st.cache.attend(q.cuda(), st.batch, workspace=ws)
            with pytest.raises(gpu_lib.BsvaError) as e:
                gpu_lib.check_status(ws)
            assert e.value.code == 6
            t.copy_(keep)
        o, ls = st.cache.attend(q.cuda(), st.batch, with_lse=True, workspace=ws)
        gpu_lib.check_status(ws)
        assert torch.equal(o, out)


def test_offsets_past_32_bits(gpu_lib):
    # a pool of more than 2^31 values, the sequence in its last pages
    H, d, page = 8, 128, 64
    n_pages = 2 ** 31 // (H * d * page) + 40
    cache = gpu_lib.PagedKVCache.over(*[torch.empty((n_pages, H, page, d), dtype=torch.int8, device="cuda") for _ in range(2)],
                                      *[torch.empty((n_pages, H, page), device="cuda") for _ in range(2)])
    rng = np.random.default_rng(51)
    i32 = dict(dtype=torch.int32, device="cuda")
    for n in (1, 150):
        k, v, q = (_bf16(rng, (200, h, d)) for h in (H, H, H))
        table = torch.arange(n_pages - 4, n_pages, **i32)[None]
        whole = gpu_lib.PagedBatch(torch.tensor([0, 200], **i32), torch.tensor([200], **i32), table, 200, 200)
        cache.write(k.cuda(), v.cuda(), whole)
        batch = gpu_lib.PagedBatch(torch.tensor([0, n], **i32), torch.tensor([200], **i32), table, n, 200)
        out, lse = cache.attend(q[:n].cuda(), batch, with_lse=True)
        kb, vb = cache.read(whole)
        for h in (0, H - 1):
            kk, vv = (paged.dequantize_rows(*paged.quantize_rows(x[:, h].float().numpy())) for x in (k, v))
            assert torch.equal(kb[0, h].cpu(), torch.from_numpy(kk).float().to(torch.bfloat16))
            close(q[:n, h].double().numpy(), kk, vv, paged.visible(n, 200), out[:, h].double().cpu().numpy(),
                  lse[:, h].double().cpu().numpy(), None, torch.int8, f"n {n} head {h}")


def test_strided_queries(gpu_lib):
    for n in (1, 60):
        st = Setup(gpu_lib, [(n, 200)], 2, 64, 16, torch.int8, seed=61)
        st.cache.write(st.new[0], st.new[1], st.batch)
        wide = _bf16(np.random.default_rng(2), (st.T, 7, 64))
        out, lse = st.cache.attend(wide.cuda()[:, 1:5], st.batch, with_lse=True)
        st.check(wide[:, 1:5], out, lse)


# ------------------------------------------------------------------------------------------ cross attention
@pytest.mark.parametrize("B,Hq,Hkv,Lq,Lk,d", [(1, 2, 2, 300, 512, 128), (3, 6, 2, 77, 33, 64), (2, 8, 1, 1, 1500, 64),
                                              (2, 3, 3, 1, 1, 128), (1, 5, 1, 1000, 130, 128), (4, 2, 1, 9, 129, 128)])
def test_cross_attention(gpu_lib, B, Hq, Hkv, Lq, Lk, d):
    rng = np.random.default_rng(Lq + Lk)
    q, k, v = _bf16(rng, (B, Hq, Lq, d)), _bf16(rng, (B, Hkv, Lk, d)), _bf16(rng, (B, Hkv, Lk, d))
    for lens in (None, [Lk, 0, Lk // 2, 1][:B], [max(1, Lk - 1), 1, 0, Lk][:B]):
        kd, vd = k.clone(), v.clone()
        for b, n in enumerate(lens or []):
            kd[b, :, n:], vd[b, :, n:] = NAN, math.inf       # what padding holds does not matter
        kl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        ws = gpu_lib.new_cross_attn_workspace(q.cuda(), kd.cuda())
        o, ls = gpu_lib.cross_attn_fwd(q.cuda(), kd.cuda(), vd.cuda(), k_len=kl, with_lse=True, workspace=ws)
        gpu_lib.check_status(ws)
        o, ls = o.double().cpu().numpy(), ls.double().cpu().numpy()
        for b in range(B):
            n = Lk if lens is None else lens[b]
            for h in range(Hq):
                hk = h // (Hq // Hkv)
                close(q[b, h].double().numpy(), k[b, hk, :n].double().numpy(), v[b, hk, :n].double().numpy(),
                      np.ones((Lq, n), bool), o[b, h], ls[b, h], None, torch.bfloat16, f"batch {b} head {h}")


# ------------------------------------------------------------------ loose bounds, many heads, repeated pages, no work
@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("max_q,max_kv", [(8, 4096), (500, 4096), (500, 100000)])
def test_bounds_far_above_the_lengths(gpu_lib, dtype, max_q, max_kv):
    # the launch follows the bounds: splits and row tiles without work; entries without tokens or pages
    lens = [(1, 70), (0, 0), (8, 8), (3, 200), (0, 40)]
    st = Setup(gpu_lib, lens, 2, 64, 16, dtype, seed=71, lead=3, tail=4)
    table = torch.full((len(lens), -(-max_kv // 16)), -1, dtype=torch.int32, device="cuda")
    table[:, :st.table.shape[1]] = st.batch.page_table
    st.batch = gpu_lib.PagedBatch(st.batch.q_start, st.batch.kv_len, table, max_q, max_kv)
    _attend(st, 6)
    _attend(st, 6, window=50)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("G", [33, 71, 128, 192])
@pytest.mark.parametrize("n", [1, 3])
def test_many_query_heads_a_key_head(gpu_lib, dtype, G, n):
    _attend(Setup(gpu_lib, [(n, 300), (1, 17)], 1, 64, 32, dtype, seed=G), G)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 70])
def test_a_page_twice_in_a_table(gpu_lib, dtype, n):
    st = Setup(gpu_lib, [(n, 200), (n, 130)], 2, 128, 32, dtype, seed=81)
    table = st.table.copy()
    table[0, 1] = table[0, 0]
    st.batch.page_table.copy_(torch.from_numpy(table))
    for z in range(2):
        st.values[z][0][32:64] = st.values[z][0][:32]
    _attend(st, 4)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 100])
def test_windows_as_long_as_the_sequences_are_none(gpu_lib, dtype, n):
    st = Setup(gpu_lib, [(n, 400), (n, n), (n, n // 2)], 2, 64, 16, dtype, seed=91)
    st.cache.write(st.new[0], st.new[1], st.batch)
    q = st.queries(4).cuda()
    a, la = st.cache.attend(q, st.batch, with_lse=True)
    for window in (400, 2 ** 30, 2 ** 31 - 1):
        b, lb = st.cache.attend(q, st.batch, window=window, with_lse=True)
        assert torch.equal(a[:2 * n], b[:2 * n]) and torch.equal(la[:2 * n], lb[:2 * n])
        assert torch.equal(torch.isinf(la), torch.isinf(lb))


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
def test_nothing_to_do(gpu_lib, dtype):
    st = Setup(gpu_lib, [(0, 20), (0, 0)], 2, 64, 16, dtype, seed=101, tail=2)
    ws = st.cache.new_workspace(st.batch, 4, st.T)
    _attend(st, 4)                                   # two rows, of no sequence: left as they were
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = st.cache.attend(q, st.batch, with_lse=True, workspace=ws)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    st.cache.write(q[:, :2], q[:, :2], st.batch, workspace=ws)
    k, v = st.cache.read(st.batch, first=torch.tensor([20, 0], dtype=torch.int32, device="cuda"), length=5, workspace=ws)
    gpu_lib.check_status(ws)
    assert (k == 0).all() and (v == 0).all()


def test_binding_refusals(gpu_lib):
    st = Setup(gpu_lib, [(1, 20)], 2, 64, 16, torch.int8, seed=5)
    b, q = st.batch, st.queries(4).cuda()
    for max_q, max_kv in ((0, 20), (2 ** 32 + 1, 20), (1, 0), (1, 2 ** 33)):
        with pytest.raises(ValueError, match="max_"):
            gpu_lib.PagedBatch(b.q_start, b.kv_len, b.page_table, max_q, max_kv)
    with pytest.raises(ValueError, match="window"):
        st.cache.attend(q, b, window=2 ** 32 + 1)
    with pytest.raises(gpu_lib.BsvaError, match="window"):
        st.cache.attend(q, b, window=-1)
    with pytest.raises(ValueError, match="shape"):
        st.cache.read(b, out=(q, q))
    with pytest.raises(TypeError):
        st.cache.attend(q.half(), b)
    with pytest.raises(ValueError, match="strides"):
        st.cache.attend(torch.zeros((1, 64, 4), dtype=torch.bfloat16, device="cuda").transpose(1, 2), b)
    with pytest.raises(ValueError, match="tokens"):
        st.cache.write(st.new[0], torch.cat([st.new[1], st.new[1]]), b)
    with pytest.raises(gpu_lib.BsvaError, match="workspace"):
        st.cache.attend(q, b, workspace=torch.zeros(255, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gpu_lib.BsvaError, match="multiple"):
        st.cache.attend(q[:, :3], b)


# ------------------------------------------------------------------------------- streams, graphs, calls at once
def _call_kinds(gpu_lib, seed):
    """A single-token call, a chunk over each kind of cache and a cross attention, as functions of their workspace."""
    kinds = []
    for dtype, lens, Hq in ((torch.int8, [(1, 900), (1, 40)], 8), (torch.int8, [(150, 700), (90, 90)], 2),
                            (torch.bfloat16, [(150, 700), (90, 90)], 2), (torch.bfloat16, [(1, 900), (1, 40)], 8)):
        st = Setup(gpu_lib, lens, 2, 64, 16, dtype, seed=seed)
        q = st.queries(Hq).cuda()
        st.cache.write(st.new[0], st.new[1], st.batch)

        def call(st=st, q=q, **kw):
            st.cache.write(st.new[0], st.new[1], st.batch, **kw)
            k, v = st.cache.read(st.batch, **kw)
            return (*st.cache.attend(q, st.batch, with_lse=True, **kw), k, v)
        kinds.append((call, st.cache.new_workspace(st.batch, Hq, st.T)))
    rng = np.random.default_rng(seed)
    for Lq in (3, 200):
        q, k, v = (_bf16(rng, (2, 4, L, 64)).cuda() for L in (Lq, 301, 301))
        kinds.append((lambda q=q, k=k, v=v, **kw: gpu_lib.cross_attn_fwd(q, k, v, with_lse=True, **kw),
                      gpu_lib.new_cross_attn_workspace(q, k)))
    return kinds


def test_given_stream_orders_what_the_call_allocates(gpu_lib):
    # on a stream that is busy, without workspace or outputs: what the call clears is cleared before its kernels
    side, busy = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    for call, ws in _call_kinds(gpu_lib, 111):
        want = call(workspace=ws)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(4):
                busy = busy @ busy * 1e-2
        got = call(stream=side)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side, workspace=ws)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_calls_at_once_on_two_streams(gpu_lib):
    kinds = [_call_kinds(gpu_lib, 121), _call_kinds(gpu_lib, 122)]
    want = [[call(workspace=ws) for call, ws in ks] for ks in kinds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [[], []]
        for i in range(len(kinds[0])):
            for z in range(2):
                j = i if z == 0 else len(kinds[0]) - 1 - i
                with torch.cuda.stream(streams[z]):
                    got[z].append((j, kinds[z][j][0](workspace=kinds[z][j][1])))
        torch.cuda.synchronize()
        for z in range(2):
            for j, g in got[z]:
                gpu_lib.check_status(kinds[z][j][1])
                assert all(torch.equal(x, y) for x, y in zip(g, want[z][j]))


def test_two_graphs_replayed_in_turn_and_at_once(gpu_lib):
    kinds = [_call_kinds(gpu_lib, 131), _call_kinds(gpu_lib, 132)]
    want = [[call(workspace=ws) for call, ws in ks] for ks in kinds]
    graphs, got = [], []
    for ks in kinds:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append([call(workspace=ws) for call, ws in ks])
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for at_once in (False, True, True):
        for outs in got:
            for o in outs:
                for x in o:
                    x.fill_(3)
        torch.cuda.synchronize()
        for z in range(2):
            with torch.cuda.stream(streams[z if at_once else 0]):
                graphs[z].replay()
        torch.cuda.synchronize()
        for z in range(2):
            for (_, ws), g, w in zip(kinds[z], got[z], want[z]):
                gpu_lib.check_status(ws)
                assert all(torch.equal(x, y) for x, y in zip(g, w))


def test_two_graphs_with_one_workspace_in_turn(gpu_lib):
    # graphs that share a workspace may follow each other on a stream: nothing is kept in it from one call for the next
    a, b = _call_kinds(gpu_lib, 141), _call_kinds(gpu_lib, 142)
    ws = torch.zeros(max(w.numel() for _, w in a + b), dtype=torch.uint8, device="cuda")
    want = [[call(workspace=ws) for call, _ in ks] for ks in (a, b)]
    graphs, got = [], []
    for ks in (a, b):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append([call(workspace=ws) for call, _ in ks])
        graphs.append(g)
    for z in (0, 1, 1, 0):
        graphs[z].replay()
    gpu_lib.check_status(ws)
    for z in range(2):
        for g, w in zip(got[z], want[z]):
            assert all(torch.equal(x, y) for x, y in zip(g, w))


# ------------------------------------------------------------- few rows: windows, joins by cluster and by kernel
@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,n,G,H", [(1, 1, 5, 1), (3, 2, 7, 1), (4, 1, 2, 6), (1, 1, 1, 2)])
@pytest.mark.parametrize("causal,window", [(True, 17), (True, 300), (True, 999), (True, 0), (False, 0)])
def test_few_rows_and_windows(gpu_lib, dtype, d, S, n, G, H, causal, window):
    # 1 to 9 splits, joined by a cluster (few CTAs) or by the second kernel; sequences much shorter than the longest
    lens = [(n, 1100), (1, 130), (0, 400), (n, 640)][:S]
    _attend(Setup(gpu_lib, lens, H, d, 32, dtype, seed=S + G), G * H, causal, window)


def test_long_sequences_of_one_head(gpu_lib):
    # more splits than a cluster joins, up to the second kernel's eight groups a row
    for n, kv in ((1, 30000), (3, 9000), (130, 20000)):
        _attend(Setup(gpu_lib, [(n, kv)], 1, 64, 256, torch.int8, seed=n), 2, window=0)
        _attend(Setup(gpu_lib, [(n, kv)], 1, 64, 256, torch.bfloat16, seed=n), 2, window=kv - 100)


def test_beside_the_block_sparse_kernel(gpu_lib):
    # both kernels hold tensor memory; on two streams at once each gives what it gives alone
    g = torch.Generator(device="cuda").manual_seed(3)
    Q, K, V = (torch.randn((1, 8, 4096, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    qk = gpu_lib.quantize_qk(Q, K)
    mask = torch.ones((1, 1, 32, 32), dtype=torch.uint8, device="cuda")

    def sparse():
        return gpu_lib.masked_block_attn_fwd(qk["q8"], qk["q_scale"], qk["k8"], qk["k_scale"], V, mask)
    kinds = _call_kinds(gpu_lib, 151)
    want, want_sparse = [call(workspace=ws) for call, ws in kinds], sparse()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for call, ws in kinds:
            with torch.cuda.stream(streams[0]):
                other = sparse()
            with torch.cuda.stream(streams[1]):
                got.append(call(workspace=ws))
        torch.cuda.synchronize()
        assert torch.equal(other, want_sparse)
        for (_, ws), x, w in zip(kinds, got, want):
            gpu_lib.check_status(ws)
            assert all(torch.equal(a, b) for a, b in zip(x, w))


# ------------------------------------------------------ several items with keys a CTA, with and without rows between them
def _check_heads(st, q, out, lse, heads, causal=True, window=0):
    G = q.shape[1] // st.H
    o_, l_ = out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
    for s, (n, kv) in enumerate(st.lens):
        ok = paged.visible(n, kv, causal, window)
        rows = slice(st.starts[s], st.starts[s] + n)
        for h in heads:
            qh, k, v = q[rows, h].double().numpy(), st.values[0][s][:, h // G], st.values[1][s][:, h // G]
            l = paged.attention_rows(qh, k, v, ok)[1] if l_ is None else l_[rows, h]
            close(qh, k, v, ok, o_[rows, h], l, None, st.dtype, f"sequence {s} head {h}")


@pytest.mark.parametrize("dtype,with_lse", [(torch.int8, True), (torch.bfloat16, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("d,G,H,window", [(128, 1, 40, 0), (64, 3, 14, 0), (64, 7, 9, 150), (128, 2, 24, 0)])
def test_many_items_a_cta(gpu_lib, dtype, with_lse, d, G, H, window):
    # 500 to 700 row tiles on 148 SMs: both halves, one half and no rows follow one another in a CTA, over odd and even
    # numbers of key tiles, so that every barrier's phase and every ring's stage meets every kind of item
    lens = [(300, 300), (100, 450), (0, 90), (257, 700), (1, 129), (300, 513), (129, 128 + 129), (40, 40)]
    st = Setup(gpu_lib, lens, H, d, 64, dtype, seed=G, tail=3)
    st.cache.write(st.new[0], st.new[1], st.batch)
    q = st.queries(G * H)
    qd, ws = q.cuda(), st.cache.new_workspace(st.batch, G * H, st.T)
    for _ in range(2):
        got = st.cache.attend(qd, st.batch, window=window, with_lse=with_lse, workspace=ws)
        out, lse = got if with_lse else (got, None)
        gpu_lib.check_status(ws)
        _check_heads(st, q, out, lse, range(0, G * H, max(1, G * H // 12)), window=window)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
def test_items_between_thousands_without_rows(gpu_lib, dtype):
    # the bound plans 24 row tiles a sequence and head where one has rows: CTAs ask for the next one many times in a row
    lens = [(1 + 7 * s % 40, 50 + 31 * s) for s in range(24)]
    st = Setup(gpu_lib, lens, 4, 64, 16, dtype, seed=161)
    st.batch = gpu_lib.PagedBatch(st.batch.q_start, st.batch.kv_len, st.batch.page_table, 3000, st.batch.max_kv)
    for _ in range(2):
        _attend(st, 8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("with_lse", [True, False])
def test_cross_attention_many_items_a_cta(gpu_lib, d, with_lse):
    B, H, Lq, Lk = 2, 40, 1100, 130
    rng = np.random.default_rng(d)
    q, k, v = _bf16(rng, (B, H, Lq, d)), _bf16(rng, (B, H, Lk, d)), _bf16(rng, (B, H, Lk, d))
    lens = [Lk, 100]
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = gpu_lib.new_cross_attn_workspace(q.cuda(), k.cuda())
    got = gpu_lib.cross_attn_fwd(q.cuda(), k.cuda(), v.cuda(), k_len=kl, with_lse=with_lse, workspace=ws)
    gpu_lib.check_status(ws)
    out, lse = got if with_lse else (got, None)
    for b, n in enumerate(lens):
        for h in range(0, H, 5):
            a = [x[b, h].double().cpu().numpy() for x in (q, k[:, :, :n], v[:, :, :n], out)]
            ok = np.ones((Lq, n), bool)
            l = paged.attention_rows(*a[:3], ok)[1] if lse is None else lse[b, h].double().cpu().numpy()
            close(*a[:3], ok, a[3], l, None, torch.bfloat16, f"batch {b} head {h}")


# --------------------------------------------------------------------------- a write that breaks a bound harms no token
@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 40])
def test_write_with_broken_lengths_leaves_the_cache(gpu_lib, dtype, n):
    # sequence 0 breaks a bound: its tokens are not written anywhere, sequence 1's are where they belong
    H, kvs = 3, (120, 64)
    broken = [("kv_len", [kvs[0] + 1, kvs[1]]), ("kv_len", [2 ** 31 - 1, kvs[1]]), ("kv_len", [-3, kvs[1]]),
              ("q_start", [-1, n, 2 * n]), ("q_start", [2 * n + 1, n, 2 * n])]
    for name, bad in broken:
        st = Setup(gpu_lib, [(n, kvs[0]), (n, kvs[1])], H, 64, 16, dtype, seed=n)
        _write_broken(gpu_lib, st, name, bad, first=1)
    # sequence 1 has more new tokens than max_q, or than there are rows
    for ends in ([0, n, 2 * n + 5], [0, n, 2 ** 31 - 1]):
        st = Setup(gpu_lib, [(n, kvs[0]), (n, kvs[1])], H, 64, 16, dtype, seed=n + 1)
        _write_broken(gpu_lib, st, "q_start", ends, first=0)


def _write_broken(gpu_lib, st, name, bad, first):
    """Writes with a broken length of the other sequence than ``first``, whose tokens alone are expected in the cache."""
    def held():
        return [x.clone().view(torch.uint8) for x in (st.cache.k, st.cache.v, st.cache.k_scale, st.cache.v_scale)
                if x is not None]
    ws = st.cache.new_workspace(st.batch, st.H, st.T)
    before = held()
    getattr(st.batch, name).copy_(torch.tensor(bad, dtype=torch.int32))
    st.cache.write(st.new[0], st.new[1], st.batch, workspace=ws)
    with pytest.raises(gpu_lib.BsvaError) as e:
        gpu_lib.check_status(ws)
    assert e.value.code == 6
    n, kv = st.lens[first]
    pages = torch.from_numpy(st.table[first][np.arange(kv - n, kv) // st.page].astype(np.int64)).unique()
    for x, y in zip(before, held()):
        keep = torch.ones(x.shape[0], dtype=torch.bool)
        keep[pages] = False
        assert torch.equal(x[keep.cuda()], y[keep.cuda()]), (name, bad)
    t = np.arange(kv)
    pg, off = st.table[first][t // st.page], t % st.page
    for z, (pool, scale) in enumerate(((st.cache.k, st.cache.k_scale), (st.cache.v, st.cache.v_scale))):
        got = pool.cpu().float().numpy()[pg, :, off]
        if st.dtype == torch.int8:
            got = got.astype(np.float64) * scale.cpu().numpy()[pg, :, off].astype(np.float64)[..., None]
        assert np.array_equal(got, st.values[z][first]), (name, bad)


# ------------------------------------------------------------------------- rows that are not a sequence's do not reach it
@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("d,G,n,window", [(64, 2, 75, 0), (128, 1, 141, 0), (128, 1, 141, 60), (64, 3, 75, 0), (64, 5, 1, 0)])
def test_other_rows_do_not_change_a_sequence(gpu_lib, dtype, d, G, n, window):
    # the queries of the next sequence and of rows behind the last one share tiles with a sequence's last rows: whatever
    # they hold, its bits stay
    st = Setup(gpu_lib, [(n, 300), (max(1, n - 34), 200)], 2, d, 16, dtype, seed=n + G, tail=50)
    st.cache.write(st.new[0], st.new[1], st.batch)
    q = st.queries(2 * G).cuda()
    want = st.cache.attend(q, st.batch, window=window, with_lse=True)
    for end in (1, 2):                 # rows before starts[end] keep their queries
        for fill in (0.0, NAN, 1e30, -1e30, math.inf):
            x = q.clone()
            x[st.starts[end]:] = fill
            got = st.cache.attend(x, st.batch, window=window, with_lse=True)
            for a, b in zip(got, want):
                assert torch.equal(a[:st.starts[end]], b[:st.starts[end]]), (end, fill)


# --------------------------------------------------------------------------------------------- NaN comes out as NaN
NAN_LENS = [[(1, 700)] * 3, [(1, 3000)] * 20, [(100, 400), (90, 90)], [(130, 4000)]]


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("lens", NAN_LENS)
def test_nan_queries_give_nan(gpu_lib, dtype, lens):
    # a diverged row must not look like one without keys (0 and -inf); the others are what they were, within the bounds
    st = Setup(gpu_lib, lens, 2, 64, 16, dtype, seed=171)
    st.cache.write(st.new[0], st.new[1], st.batch)
    q = st.queries(4)
    at = [(0, 1), (st.T // 2, 3), (st.T - 1, 0)]
    bad = q.clone()
    for t, h in at:
        bad[t, h, 5] = NAN
    out, lse = st.cache.attend(bad.cuda(), st.batch, with_lse=True)
    for t, h in at:
        assert torch.isnan(out[t, h]).all() and torch.isnan(lse[t, h])
    good = st.cache.attend(q.cuda(), st.batch, with_lse=True)
    for t, h in at:
        out[t, h], lse[t, h] = good[0][t, h], good[1][t, h]
    st.check(q, out, lse)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("lens", NAN_LENS)
def test_nan_keys_give_nan(gpu_lib, dtype, lens):
    # every row that sees the key
    st = Setup(gpu_lib, lens, 2, 64, 16, dtype, seed=181)
    st.cache.write(st.new[0], st.new[1], st.batch)
    q = st.queries(4).cuda()
    for t in (0, min(n for n, _ in lens) // 2 + 20):
        for h in range(2):
            pool = st.cache.k_scale if dtype == torch.int8 else st.cache.k
            row = pool[st.table[0][t // 16], h, t % 16]
            keep = row.clone()
            row.fill_(NAN)
            out, lse = st.cache.attend(q, st.batch, with_lse=True)
            row.copy_(keep)
            n, kv = lens[0]
            rows = slice(max(0, t - (kv - n)), n)
            assert torch.isnan(out[rows, 2 * h:2 * h + 2]).all() and torch.isnan(lse[rows, 2 * h:2 * h + 2]).all()


def test_nan_queries_in_cross_attention(gpu_lib):
    for Lq in (3, 200):
        q, k, v = (torch.ones((1, 2, L, 64), dtype=torch.bfloat16, device="cuda") for L in (Lq, 300, 300))
        q[0, 1, Lq - 1, 0] = NAN
        out, lse = gpu_lib.cross_attn_fwd(q, k, v, with_lse=True)
        assert torch.isnan(out[0, 1, Lq - 1]).all() and torch.isnan(lse[0, 1, Lq - 1])
        assert (out[0, 0] == 1).all() and (out[0, 1, :Lq - 1] == 1).all()


# ------------------------------------------------------------------------------- values up to the largest finite ones
@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[(1, 700)] * 3, [(1, 3000)] * 20, [(1, 9)], [(100, 400), (90, 90)], [(130, 4000)]])
def test_the_largest_values(gpu_lib, dtype, d, lens):
    # values of 2^126 to 2^127: a weighted mean is finite, a sum of two is not; all of one sign, so that no error hides
    st = Setup(gpu_lib, lens, 2, d, 16, dtype, seed=191)
    for s, (n, kv) in enumerate(lens):
        x = (1 + torch.rand((kv, 2, d), generator=torch.Generator().manual_seed(s))).mul(2.0 ** 126).to(torch.bfloat16)
        codes, sc = paged.quantize_rows(x.float().numpy())
        st.values[1][s] = paged.dequantize_rows(codes, sc) if dtype == torch.int8 else x.double().numpy()
        t = np.arange(kv)
        pg = torch.from_numpy(st.table[s][t // 16].astype(np.int64)).cuda()
        off = torch.from_numpy(t % 16).cuda()
        if dtype == torch.int8:
            st.cache.v[pg, :, off] = torch.from_numpy(codes).cuda()
            st.cache.v_scale[pg, :, off] = torch.from_numpy(sc).cuda()
        else:
            st.cache.v[pg, :, off] = x.cuda()
        if n:
            st.new[1][st.starts[s]:st.starts[s + 1]] = x[kv - n:].cuda()
    _attend(st, 4)
    _attend(st, 4, qscale=20.0)


@pytest.mark.parametrize("Lq", [1, 300])
def test_the_largest_values_in_cross_attention(gpu_lib, Lq):
    g = torch.Generator().manual_seed(Lq)
    q, k = (torch.randn((2, 2, L, 64), generator=g).to(torch.bfloat16) for L in (Lq, 500))
    v = (1 + torch.rand((2, 2, 500, 64), generator=g)).mul(2.0 ** 126).to(torch.bfloat16)
    out, lse = gpu_lib.cross_attn_fwd(q.cuda(), k.cuda(), v.cuda(), with_lse=True)
    for b in range(2):
        for h in range(2):
            close(*[x[b, h].double().numpy() for x in (q, k, v)], np.ones((Lq, 500), bool), out[b, h].double().cpu().numpy(),
                  lse[b, h].double().cpu().numpy(), None, torch.bfloat16, f"batch {b} head {h}")


@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16])
@pytest.mark.parametrize("lens", [[(1, 700)] * 3, [(1, 3000)] * 20, [(100, 400), (90, 90)], [(130, 4000)]])
def test_values_of_small_magnitude(gpu_lib, dtype, lens):
    # all values times 2^-50 (exact): outputs are what they are at ordinary magnitudes, times 2^-50, within the bounds
    st = Setup(gpu_lib, lens, 2, 64, 16, dtype, seed=201, mag=0.3)
    (st.cache.v_scale if dtype == torch.int8 else st.cache.v).mul_(2.0 ** -50)
    st.new[1].mul_(2.0 ** -50)
    st.values[1] = [x * 2.0 ** -50 for x in st.values[1]]
    _attend(st, 4)


def test_the_largest_values_under_weights_above_the_first_maximum(gpu_lib):
    # the first keys' logits are 33 powers of two below all others': their maximum is kept, each later key weighs 2^33, and
    # their sum over one long pass (as many row tiles as SMs: no splits) must not reach the top of fp32
    Lq, Lk, d = 256 * 148, 50000, 64
    q, k, v = (torch.zeros((1, 1, L, d), dtype=torch.bfloat16, device="cuda") for L in (Lq, Lk, Lk))
    q[..., 0], k[0, 0, 64:, 0] = 1.0, 22.75
    v[:] = (1 + torch.rand((Lk, 1), generator=torch.Generator().manual_seed(1))).mul(2.0 ** 126).to(torch.bfloat16).cuda()
    out, lse = gpu_lib.cross_attn_fwd(q, k, v, softmax_scale=1.0, with_lse=True)
    assert (out == out[:, :, :1]).all() and (lse == lse[:, :, :1]).all()
    close(*[x[0, 0, :1].double().cpu().numpy() if x is q else x[0, 0].double().cpu().numpy() for x in (q, k, v)],
          np.ones((1, Lk), bool), out[0, 0, :1].double().cpu().numpy(), lse[0, 0, :1].double().cpu().numpy(), 1.0,
          torch.bfloat16, "first row")


# -------------------------------------------------------------- one token whose values are far larger than the others'
@pytest.mark.parametrize("lens,page,window,big", [
    ([(200, 200)], 16, 0, 199),          # tiles: only the last row sees it, those before share its tile of rows and keys
    ([(200, 460)], 64, 0, 455),
    ([(130, 300)], 16, 90, 82),          # at the first rows' end of the window: gone for the later ones
    ([(10, 300)], 16, 0, 299),           # few rows
    ([(10, 10)], 16, 0, 9),
    ([(10, 300)], 16, 40, 252),
    ([(1, 300)], 16, 0, 150)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [8, 12, 16])
def test_small_values_beside_a_large_one(gpu_lib, lens, page, window, big, d, power):
    """INT8. A row's bound has only what it sees in it, but for the steps of f16 below 2^-14, which are relative to the
    largest scale S that its tile of rows meets: R = S / s for a visible scale s.

    Tiles: a value enters as code * f, f = s c with 2^5 <= S c < 2^8, so f >= 2^5 / R >= 2^-14 for R <= 2^19: f and the
    product round within 2^-11 each, but for products below 2^-14 that lose 2^-25, 2^-25 / c <= 2^-30 S of a value.
    A weight rounds within 2^-11, or by 2^-25 below 2^-14 (n 2^-25 max|v| over the visible keys; relative to a largest
    weight of at least 1).
    Few rows: a weight enters as p s c with 2^6 <= S c < 2^7, rounded within 2^-11, or below 2^-14 by at most 2^-25 and
    never by more than itself: of p s that is min(2^-31 S, p s), times codes of at most 127."""
    (n, kv), H, G = lens[0], 1, 2
    st = Setup(gpu_lib, lens, H, d, page, torch.int8, seed=power, mag=0.3)
    x = st.kv[1][0]
    x[big] *= 2.0 ** power
    codes, sc = paged.quantize_rows(x.float().numpy())
    st.values[1][0] = paged.dequantize_rows(codes, sc)
    t = np.arange(kv)
    pg, off = torch.from_numpy(st.table[0][t // page].astype(np.int64)).cuda(), torch.from_numpy(t % page).cuda()
    st.cache.v[pg, :, off] = torch.from_numpy(codes).cuda()
    st.cache.v_scale[pg, :, off] = torch.from_numpy(sc).cuda()
    st.cache.write(st.new[0], x[kv - n:].cuda(), st.batch)
    q = st.queries(G)
    ws = st.cache.new_workspace(st.batch, G, st.T)
    out, _ = st.cache.attend(q.cuda(), st.batch, window=window, with_lse=True, workspace=ws)
    gpu_lib.check_status(ws)
    out = out.double().cpu().numpy()
    ok = paged.visible(n, kv, True, window)
    k, v = st.values[0][0][:, 0], st.values[1][0][:, 0]
    s, S = sc[:, 0].astype(np.float64), float(sc.max())
    for h in range(G):
        qh = q[:, h].double().numpy()
        ro, _, A = paged.attention_rows(qh, k, v, ok)
        logit = np.where(ok, qh @ k.T / math.sqrt(d), -np.inf)
        p = np.exp(logit - logit.max(1, keepdims=True))
        dx = ((d + 4) * 2.0 ** -24 / math.sqrt(d) * np.where(ok, np.abs(qh) @ np.abs(k).T, 0).max(1))[:, None]
        vmax = np.where(ok, np.abs(v).max(1), 0).max(1)[:, None]
        tol = 2.0 ** -8 * np.abs(ro) + (3 * 2.0 ** -11 + 4 * dx + (kv + 8) * 2.0 ** -22) * A * 1.01
        if n * G > 64:
            tol += kv * 2.0 ** -25 * vmax + 2.0 ** -30 * S
        else:
            tol += (127 * np.minimum(2.0 ** -31 * S, p * s).sum(1) / p.sum(1))[:, None]
        worst = (np.abs(out[:, h] - ro) / tol).max()
        assert worst <= 1, f"head {h}: {worst} of the bound"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fill", [NAN, math.inf, -math.inf])
def test_values_that_are_not_finite_read_back_as_nan(gpu_lib, d, fill):
    # wherever in the row they are; the other rows are what they are without
    st = Setup(gpu_lib, [(150, 150), (5, 40)], 2, d, 16, torch.int8, seed=d)
    st.cache.write(st.new[0], st.new[1], st.batch)
    want = st.cache.read(st.batch)
    k, v = (x.clone() for x in st.new)
    bad = torch.zeros((2, st.T, 2), dtype=torch.bool)
    for i in range(d):
        for z, x in enumerate((k, v)):
            x[(i + z) % 150, i % 2, i] = fill
            bad[z, (i + z) % 150, i % 2] = True
    st.cache.write(k, v, st.batch)
    got = st.cache.read(st.batch)
    for z in range(2):
        b = bad[z, :150].T.cuda()
        assert torch.isnan(got[z][0, :, :150][b]).all() and torch.equal(got[z][0, :, :150][~b], want[z][0, :, :150][~b])
        assert torch.equal(got[z][1], want[z][1])
    for n in (1, 150):        # the last rows see every key: NaN wherever a key or value of their head is bad
        batch = gpu_lib.PagedBatch(torch.tensor([0, n, n], dtype=torch.int32, device="cuda"), st.batch.kv_len,
                                   st.batch.page_table, n, 150)
        out = st.cache.attend(torch.ones((n, 2, d), dtype=torch.bfloat16, device="cuda"), batch)
        assert torch.isnan(out[n - 1]).all()


@pytest.mark.parametrize("dtype,power", [(torch.int8, -100), (torch.int8, 117), (torch.bfloat16, -90), (torch.bfloat16, 90)])
@pytest.mark.parametrize("n", [1, 5, 80])
def test_queries_and_keys_far_from_one(gpu_lib, dtype, n, power):
    # queries times 2^power, keys times 2^-power: the same logits. Powers of two are exact everywhere, so are the bits
    st = Setup(gpu_lib, [(n, 300)], 2, 64, 16, dtype, seed=n, mag=0.3)
    st.cache.write(st.new[0], st.new[1], st.batch)
    q = st.queries(4).clamp(-0.9, 0.9).cuda()
    want = st.cache.attend(q, st.batch, with_lse=True)
    (st.cache.k_scale if dtype == torch.int8 else st.cache.k).mul_(2.0 ** -power)
    got = st.cache.attend(q * 2.0 ** power, st.batch, with_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_numbers_past_32_bits_are_refused(gpu_lib):
    # nothing wraps on its way into the C entries
    st = Setup(gpu_lib, [(1, 20)] * 130, 2, 64, 16, torch.int8, seed=5)
    b, q = st.batch, st.queries(4).cuda()
    for window in (-2 ** 31 - 1, -2 ** 32 + 5, 2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError, match="window"):
            st.cache.attend(q, b, window=window)
    loose = gpu_lib.PagedBatch(b.q_start, b.kv_len, b.page_table, 2 ** 24, 20)
    with pytest.raises(ValueError, match="packed rows"):     # the default, S * max_q, is 130 * 2^24
        st.cache.new_workspace(loose, 4)
    ws = st.cache.new_workspace(loose, 4, st.T)
    st.cache.write(st.new[0], st.new[1], loose, workspace=ws)
    gpu_lib.check_status(ws)
