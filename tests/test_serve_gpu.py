"""The operators of include/qsa_serve.h on the GPU against their definitions in
64 bits (tests/_serve_ref.py). Tolerances: see attn_tol and weights there;
positions, counts, tokens and copied rows are equal."""

import math

import numpy as np
import pytest
import torch

from tests import _kv_ref as R
from tests import _serve_ref as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import __graft_entry__

    __graft_entry__.build()
    from block_sparse_attention_qsa_gb300 import qsa as q

    return q


def _ok(qsa, ws):
    st, info = qsa.check_errors(ws)
    assert st == qsa.OK, info


def _normal(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _i32(a):
    return torch.tensor(a, dtype=torch.int32).cuda()


def _up(table, n):
    """The pages n further on (entries that are none stay)."""
    return torch.where(table >= 0, table + n, table)


def _dims(qsa, B, max_pages, num_pages, kv="bf16", n_q=1, hq=16, hk=2, D=128, ps=64, **kw):
    return qsa.make_dims(B, n_q, max(1, max_pages * ps // 4), max_pages, num_pages, 1, kv, ps, hq, hk, D, **kw)


# --------------------------------------------------------------------------
# attention over a shared prefix
# --------------------------------------------------------------------------
GARBAGE = (-7, 1 << 30, -1, 2 ** 31 - 1)


class Prefixed:
    """A batch over `prefix` shared pages with own[r] tokens behind them."""

    def __init__(self, qsa, prefix, own, n_q=1, hq=16, hk=2, D=128, ps=64, kv="bf16", q_pos=None, seed=11, mutate=None,
                 sm_scale=0.0, extra_pages=0):
        B = len(own)
        shared_table, n_shared = R.page_table([max(1, prefix * ps)], ps, seed, spare=0)
        table, n_own = R.page_table([max(1, c) for c in own], ps, seed + 1)
        self.prefix = shared_table[0, :prefix].clone()
        own_table = table + n_shared
        own_table[table < 0] = -1
        junk = torch.tensor([[GARBAGE[(r + i) % 4] for i in range(prefix)] for r in range(B)], dtype=torch.int32)
        self.table = torch.cat([junk.view(B, prefix), own_table], 1).to(torch.int32).contiguous()
        if extra_pages:
            self.table = torch.nn.functional.pad(self.table, (0, extra_pages), value=-7)
        self.full = torch.cat([self.prefix.expand(B, -1), self.table[:, prefix:]], 1)
        num_pages = n_shared + n_own
        self.kc, self.vc, self.ks, self.vs = R.make_cache(num_pages, hk, ps, D, kv, seed + 2)
        self.q = _normal((B, n_q, hq, D), seed + 3)
        L = prefix * ps
        if q_pos is None:
            q_pos = [[max(-1, L + c - n_q + j) for j in range(n_q)] for c in own]
        self.q_pos = np.array(q_pos, dtype=np.int32)
        if mutate:
            mutate(self)
        self.kv, self.B, self.n_q, self.L = kv, B, n_q, L
        self.d = _dims(qsa, B, self.table.shape[1], num_pages, kv, n_q, hq, hk, D, ps, sm_scale=sm_scale)
        self.ws = qsa.make_prefix_workspace(self.d, prefix)
        self.out = torch.full((B, n_q, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((B, n_q, hq), 7.0, device="cuda")
        self.args = (self.d, self.q, self.kc, self.vc, self.ks, self.vs, self.prefix.cuda(), self.table.cuda(),
                     _i32(self.q_pos.tolist()), self.out, self.ws)

    def run(self, qsa, alone=None, **kw):
        """alone: None as prefix_attn chooses, else as told."""
        if alone is None:
            qsa.prefix_attn(*self.args, lse=self.lse, **kw)
        else:
            qsa.test_prefix_attn(*self.args, lse=self.lse, alone=alone, **kw)
        return self

    def compare(self, skip=(), gone=None):
        """gone: positions left out, of every request."""
        d = self.d
        sc = [R.f64(s)[None, :, None] if self.kv == "fp8" else 1.0 for s in (self.ks, self.vs)]
        caches = [R.f64(self.kc), R.f64(self.vc)]
        full, q64, got, got_lse = self.full.numpy(), R.f64(self.q), R.f64(self.out), R.f64(self.lse)
        scale = d.sm_scale if d.sm_scale > 0 else 1.0 / math.sqrt(d.head_dim)
        cap = d.max_pages * d.page_size
        for r in range(self.B):
            top = max([int(p) for p in self.q_pos[r] if 0 <= p < cap], default=-1) + 1
            if top:
                k, v = (R.rows(c, full[r], top) * s for c, s in zip(caches, sc))
            for j in range(self.n_q):
                p = int(self.q_pos[r, j])
                if (r, j) in skip:
                    continue
                if p < 0 or p >= cap:
                    assert np.all(got[r, j] == 0) and np.all(got_lse[r, j] == -np.inf), (r, j)
                    continue
                see = np.arange(p + 1) if gone is None else np.setdiff1d(np.arange(p + 1), gone)
                ref, rl, mag, qk, small = R.attention(q64[r, j], k[see], v[see], scale, 0, len(see))
                tol, tol_l = S.attn_tol(ref, mag, rl, qk, d.head_dim, self.kv, small)
                err, err_l = np.abs(got[r, j] - ref), np.abs(got_lse[r, j] - rl)
                assert np.all(err <= tol), (r, j, err.max(), (err - tol).max())
                assert np.all(err_l <= tol_l), (r, j, err_l.max())
        return self


def _prefix_case(qsa, *a, **kw):
    """The prefix read once for all requests, and by each for itself; what
    prefix_attn chooses is one of the two, bit for bit."""
    c = Prefixed(qsa, *a, **kw)
    both = []
    for alone in (True, False):
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        c.run(qsa, alone=alone)
        _ok(qsa, c.ws)
        c.compare()
        both.append((c.out.clone(), c.lse.clone()))
    c.run(qsa)
    _ok(qsa, c.ws)
    assert any(torch.equal(c.out, o) and torch.equal(c.lse, l) for o, l in both)
    c.out.copy_(both[1][0])
    c.lse.copy_(both[1][1])
    return c


HEADS = [(16, 2, 128), (8, 1, 64), (4, 4, 256), (12, 4, 64), (7, 1, 128), (32, 2, 128), (24, 1, 256), (40, 1, 64)]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hk,D", HEADS)
@pytest.mark.parametrize("n_q", [1, 4])
def test_prefix_heads(qsa, kv, hq, hk, D, n_q):
    _prefix_case(qsa, 9, [5, 70, 4, 300, 64, 129, 6], n_q, hq, hk, D, 64, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("prefix", [1, 7, 33])
def test_prefix_lengths(qsa, kv, ps, prefix):
    _prefix_case(qsa, prefix, [1, 2, ps, ps + 1, 3 * ps - 1], 1, 8, 2, 128, ps, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_queries_anywhere(qsa, kv, D):
    # padding, queries that see no own token, that see a part of the prefix only, in any order, and both in a request
    L = 5 * 32
    pos = [[-1, -1, -1, -1], [L - 1, L - 1, L - 1, L - 1], [L - 1, L, L + 1, L + 2], [L - 2, L - 1, L, L + 1],
           [0, 1, 2, 3], [L + 40, 3, L + 7, -1], [-1, L + 5, -1, L - 1], [L + 90, L + 91, L + 92, L + 93], [0, -1, -1, -1]]
    _prefix_case(qsa, 5, [94] * len(pos), 4, 16, 2, D, 32, kv, q_pos=pos)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_all_padding_and_all_apart(qsa, kv):
    _prefix_case(qsa, 4, [10] * 3, 2, q_pos=[[-1, -1]] * 3, kv=kv)
    _prefix_case(qsa, 4, [10] * 3, 2, q_pos=[[100, 7], [0, 1], [253, 254]], kv=kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("prefix,own,n_q", [(313, [1, 900], 4), (157, [33] * 40, 1), (641, [3, 5000, 1], 1), (40, [70] * 20, 4),
                                            (391, [5, 64, 300], 4)])
def test_prefix_long_and_wide(qsa, kv, prefix, own, n_q):
    _prefix_case(qsa, prefix, own, n_q, kv=kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_long_parts(qsa, kv, D):
    # many heads: few parts of the prefix each, so that a CTA's ring of tiles goes round several times
    _prefix_case(qsa, 40, [3] * 17, 1, 640, 80, D, 64, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_long_own_positions(qsa, kv):
    # one CTA has all 259 tiles of a request's own positions, more than an accumulator in tensor memory holds at
    # once; the requests' tables name the same pages
    B = 152
    c = Prefixed(qsa, 4, [259 * 128 - 5], 1, 1, 1, 64, kv=kv)
    c.B, c.q = B, _normal((B, 1, 1, 64), 5)
    c.q_pos, c.full = np.repeat(c.q_pos, B, 0), c.full.expand(B, -1)
    c.d = _dims(qsa, B, c.table.shape[1], c.d.num_pages, kv, 1, 1, 1, 64)
    c.ws = qsa.make_prefix_workspace(c.d, 4)
    c.out = torch.full((B, 1, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    c.lse = torch.full((B, 1, 1), 7.0, device="cuda")
    c.args = (c.d, c.q, *c.args[2:7], c.table.expand(B, -1).contiguous().cuda(), _i32(c.q_pos.tolist()), c.out, c.ws)
    c.run(qsa, alone=False)
    _ok(qsa, c.ws)
    c.compare()


@pytest.mark.parametrize("D,B,hq,hk", [(128, 300, 8, 1), (64, 700, 4, 2), (256, 257, 4, 1)])
def test_prefix_many_requests(qsa, D, B, hq, hk):
    rng = np.random.RandomState(3)
    _prefix_case(qsa, 9, [int(x) for x in rng.randint(1, 60, B)], 1, hq, hk, D, 16)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hk,n_q", [(1024, 1, 2), (64, 64, 3), (129, 1, 1), (3, 3, 1)])
def test_prefix_head_counts(qsa, kv, hq, hk, n_q):
    _prefix_case(qsa, 11, [4, 90], n_q, hq, hk, 64, 16, kv)


def test_prefix_of_no_pages_is_paged_attn(qsa):
    c = _prefix_case(qsa, 0, [100, 7, 333], 2)
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    qsa.paged_attn(c.d, c.q, c.kc, c.vc, c.ks, c.vs, c.args[7], c.args[8], out, c.ws, lse=lse)
    assert torch.equal(out, c.out) and torch.equal(lse, c.lse)


def test_prefix_of_every_page(qsa):
    # the whole table is shared
    c = Prefixed(qsa, 8, [1, 1, 1], 2, ps=16, q_pos=[[126, 127], [127, 127], [3, -1]])
    table = c.table[:, :8].contiguous()
    d = _dims(qsa, 3, 8, c.d.num_pages, "bf16", 2, ps=16)
    ws = qsa.make_prefix_workspace(d, 8)
    c.d = d
    for alone in (False, True):
        qsa.test_prefix_attn(d, *c.args[1:7], table.cuda(), c.args[8], c.out, ws, lse=c.lse, alone=alone)
        _ok(qsa, ws)
        c.compare()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("sm_scale", [1e-3, 2.0])
def test_prefix_scale(qsa, kv, sm_scale):
    _prefix_case(qsa, 20, [90, 5], 4, kv=kv, sm_scale=sm_scale)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("factor", [1e5, 1e-6])
def test_prefix_query_magnitudes(qsa, kv, factor):
    def scale_q(c):
        c.q.mul_(factor)
    _prefix_case(qsa, 20, [90, 5], 4, kv=kv, sm_scale=0.05 / factor, mutate=scale_q)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_what_is_masked_never_arrives(qsa, kv, bad, D):
    # every slot that no query sees is NaN or infinite, and in requests that
    # see a part of the prefix, nothing behind their queries arrives
    if kv == "fp8" and not math.isnan(bad):
        pytest.skip("E4M3 has no infinities")
    code = torch.tensor(bad).to(torch.bfloat16) if kv == "bf16" else 0x7F
    ps, L = 16, 9 * 16
    own = [77, 3, 130]
    pos = [[L + c - 2, L + c - 1] for c in own]

    def poison(c):
        seen = torch.zeros(c.kc.shape[0], ps, dtype=torch.bool)
        for r, n in enumerate(own):
            p = np.arange(L + n)
            seen[torch.from_numpy(c.full.numpy()[r, p // ps].astype(np.int64)), torch.from_numpy(p % ps)] = True
        for x in (c.kc, c.vc):
            x.transpose(1, 2)[~seen.cuda()] = code

    c = _prefix_case(qsa, 9, own, 2, 16, 2, D, ps, kv, q_pos=pos, mutate=poison)
    # a poisoned position of the prefix: only requests that see less keep clear of it
    c.q_pos[1] = [50, 52]
    c.args[8].copy_(_i32(c.q_pos.tolist()))
    page, slot = int(c.prefix[3]), 5  # position 53
    for x in (c.kc, c.vc):
        x[page, :, slot] = code
    for alone in (True, False):
        c.run(qsa, alone=alone)
        _ok(qsa, c.ws)
        c.compare(skip=[(0, 0), (0, 1), (2, 0), (2, 1)])
        assert torch.isnan(c.out[0].float()).all() and torch.isnan(c.out[2].float()).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_prefix_not_finite_queries_stay_in_their_rows(qsa, kv, bad):
    def poison(c):
        c.q[1, 0, 5, 7] = bad
        c.q[3] = bad
    c = Prefixed(qsa, 10, [30, 4, 9, 2], 2, kv=kv, mutate=poison,
                 q_pos=[[668, 669], [642, 643], [647, 648], [-1, -1]])
    q = c.q.clone()
    good = [h for h in range(16) if h != 5]
    for alone in (True, False):
        c.q.copy_(q)
        c.run(qsa, alone=alone)
        _ok(qsa, c.ws)
        assert torch.isnan(c.out[1, 0, 5].float()).all()
        first = c.out[1, 0, good].clone()
        c.q[1, 0, 5] = 0
        c.q[3] = 0
        c.compare(skip=[(1, 0)])
        c.q[1, 0, 5] = 1
        c.q[3] = 1
        c.run(qsa, alone=alone)
        assert torch.equal(c.out[1, 0, good], first)


def test_prefix_infinite_values_arrive(qsa):
    def poison(c):
        c.vc[int(c.prefix[2]), 0, 1, 3] = math.inf
        c.vc[int(c.prefix[2]), 1, 1, 4] = -math.inf
    c = Prefixed(qsa, 6, [9, 1], 1, mutate=poison)
    for alone in (True, False):
        c.run(qsa, alone=alone)
        _ok(qsa, c.ws)
        out = c.out.float()
        assert (out[:, :, :8, 3] == math.inf).all() and (out[:, :, 8:, 4] == -math.inf).all()
        out[:, :, :8, 3] = out[:, :, 8:, 4] = 0
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
def test_prefix_one_key_far_above(qsa, kv, D):
    # the largest scores come late, early, or in the own part: 40 to 200 above the others
    def spread(c):
        for i, (page, up) in enumerate([(17, 3.0), (2, 4.0), (19, 6.0)]):
            c.kc[int(c.prefix[page]), :, 5 + i] = c.q[0, 0, 0].mul(up) if kv == "bf16" else \
                (c.q[0, 0, 0].float() * up / c.ks[0]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    _prefix_case(qsa, 20, [90, 5], 2, 4, 1, D, kv=kv, mutate=spread)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("rate", [0.02, 0.2, 1.5, -0.2])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_rising_scores(qsa, kv, rate, D):
    # scores that rise (or fall) by `rate` a position: references move between tiles, and within them
    def ramp(c):
        t = torch.arange(c.full.shape[1] * 32, device="cuda").float()
        for r in range(c.full.shape[0]):
            row = c.full[r].long().cuda()
            ok = row >= 0
            k = torch.zeros((c.full.shape[1], 32, D), device="cuda")
            k[..., 3] = (t * rate if rate > 0 else (t - 700) * rate).view(-1, 32)
            if kv == "fp8":  # (a code's value times its scale)
                k = (k / c.ks[0]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                k = k.to(torch.bfloat16)
            c.kc[row[ok], 0] = k[ok]
        c.q.zero_()
        c.q[..., 3] = 1.0
    _prefix_case(qsa, 22, [90, 5, 33], 2, 4, 1, D, 32, kv=kv, mutate=ramp, sm_scale=1.0)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("up", [10, 24, 30, 60])
def test_prefix_huge_equal_scores(qsa, kv, up):
    # every score is 2^up or so: the weights are equal, the output is the mean of V and lse is near the score
    def flat(c):
        c.q.fill_(2.0 ** (up - 7))
        c.kc.fill_(1.0) if kv == "bf16" else c.kc.fill_(0x38)
        c.ks.fill_(1.0)
    c = Prefixed(qsa, 22, [90, 5, 33], 2, 4, 1, 128, 32, kv=kv, mutate=flat, sm_scale=1.0)
    for alone in (True, False):
        c.run(qsa, alone=alone)
        _ok(qsa, c.ws)
        v = R.f64(c.vc) * (float(c.vs[0]) if kv == "fp8" else 1.0)
        for r in range(3):
            for j in range(2):
                rows = R.rows(v, c.full.numpy()[r], int(c.q_pos[r, j]) + 1)[:, 0]
                ref, mag = rows.mean(0), np.abs(rows).mean(0)
                tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -18) * mag
                assert np.all(np.abs(R.f64(c.out)[r, j] - ref) <= tol), (alone, r, j)
                assert np.allclose(R.f64(c.lse)[r, j], 2.0 ** up + math.log(len(rows)), rtol=2.0 ** -20)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_lowest_scores(qsa, kv):
    # every score is far below 0, or -infinity (BF16)
    def low(c):
        c.q.fill_(-20.0)
        c.kc.fill_(60.0) if kv == "bf16" else c.kc.fill_(0x70)
    _prefix_case(qsa, 6, [40, 3], 2, kv=kv, mutate=low)
    if kv == "bf16":
        def lowest(c):
            c.q.fill_(-1.0)
            c.kc.fill_(math.inf)
        c = Prefixed(qsa, 6, [40, 3], 2, mutate=lowest)
        for alone in (True, False):
            c.run(qsa, alone=alone)
            _ok(qsa, c.ws)
            assert (c.out == 0).all() and (c.lse == -math.inf).all()


@pytest.mark.parametrize("kv,D,T", [("bf16", 128, 300000), ("fp8", 128, 300000), ("bf16", 64, 1000000), ("fp8", 64, 260000)])
def test_prefix_long_sums(qsa, kv, D, T):
    # equal keys: the output is the mean of V. V is 1 everywhere: off by the
    # accumulators' cutting (2^-12),
    # the weights' rounding (equal weights: 2^-8 all in one direction) and the
    # result's (2^-8); lse is ln T within 2^-18 of itself and as much
    ps = 256
    pages = T // ps
    kc = torch.zeros((3, 1, ps, D), dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
    vc = torch.full_like(kc, 1.0) if kv == "bf16" else torch.full_like(kc, 0x38)
    one = torch.ones(1, device="cuda")
    d = _dims(qsa, 2, pages + 1, 3, kv, 1, 4, 1, D, ps)
    ws = qsa.make_prefix_workspace(d, pages)
    shared = torch.arange(pages, dtype=torch.int32, device="cuda") % 2
    table = torch.full((2, pages + 1), 2, dtype=torch.int32, device="cuda")
    q = _normal((2, 1, 4, D), 5)
    out, lse = torch.empty_like(q), torch.empty((2, 1, 4), device="cuda")
    pos = _i32([[pages * ps + 9], [pages * ps - 1]])
    qsa.test_prefix_attn(d, q, kc, vc, one, one, shared, table, pos, out, ws, lse=lse)
    _ok(qsa, ws)
    assert (out.float() - 1).abs().max().item() <= 2.0 ** -7 + 2.0 ** -12
    want = torch.log((pos.double() + 1)).unsqueeze(-1)
    assert (lse.double() - want).abs().max().item() <= 2.0 ** -18 * (1 + math.log(T))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("alone", [True, False])
def test_prefix_reports_bad_pages(qsa, kv, alone):
    c = Prefixed(qsa, 12, [50, 9], 2, ps=32, kv=kv)
    for bad in (-1, c.d.num_pages, 2 ** 31 - 1):
        t = c.args[6]
        t.copy_(c.prefix)
        t[7] = bad
        c.run(qsa, alone=alone)
        st, info = qsa.check_errors(c.ws)
        assert st == qsa.ERR_BAD_INDEX and info == (2, -1, 0, bad)
        c.compare(gone=np.arange(7 * 32, 8 * 32))
    c.args[6].copy_(c.prefix)
    own = c.args[7].clone()
    c.args[7][1, 12] = -3  # request 1's own page
    c.run(qsa, alone=alone)
    st, info = qsa.check_errors(c.ws)
    assert st == qsa.ERR_BAD_INDEX and info == (2, 1, 0, -3)
    c.compare(skip=[(1, 0), (1, 1)])
    c.args[7].copy_(own)
    # every page of the prefix is bad: what is left is the own part
    c.args[6].fill_(-1)
    c.run(qsa, alone=alone)
    assert qsa.check_errors(c.ws)[0] == qsa.ERR_BAD_INDEX
    c.compare(gone=np.arange(12 * 32))
    c.args[6].copy_(c.prefix)
    c.args[8][0, 1] = c.d.max_pages * 32  # past the table
    c.q_pos[0, 1] = c.d.max_pages * 32
    c.run(qsa, alone=alone)
    st, info = qsa.check_errors(c.ws)
    assert st == qsa.ERR_BAD_INDEX and info == (1, 0, 1, c.d.max_pages * 32)
    c.compare()


@pytest.mark.parametrize("kv,prefix,own,n_q", [("bf16", 100, [70, 1, 300], 4), ("fp8", 313, [900] * 9, 1), ("bf16", 5, [3] * 60, 2)])
def test_prefix_same_bits_streams_and_graphs(qsa, kv, prefix, own, n_q):
    c = _prefix_case(qsa, prefix, own, n_q, kv=kv)
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.out.zero_()
        c.run(qsa, alone=False)
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    qsa.test_prefix_attn(*c.args)  # without lse
    assert torch.equal(c.out, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = Prefixed(qsa, prefix, own, n_q, kv=kv, seed=99)
    other.ws = c.ws
    other.args = other.args[:-1] + (c.ws,)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, x in zip(graphs, (c, other)):
        with torch.cuda.graph(g, stream=side):
            x.run(qsa, alone=False)
    # two graphs that share a workspace, replayed in turn, and eager calls between
    for _ in range(3):
        c.out.zero_()
        other.out.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, out)
        other.compare()
    c.out.zero_()
    c.run(qsa, alone=False, stream=side)
    side.synchronize()
    assert torch.equal(c.out, out)
    # back to back with no wait between: the pieces of one are not another's
    outs = []
    for x in (c, other, c, other):
        y = torch.empty_like(x.out)
        qsa.test_prefix_attn(*x.args[:9], y, c.ws)
        outs.append(y)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[2], out) and torch.equal(outs[1], outs[3])
    assert torch.equal(outs[1], other.out)
    _ok(qsa, c.ws)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_offsets_past_32_bits(qsa, kv):
    ps, hk, D = 64, 2, 128
    num_pages = (1 << 31) // (ps * hk * D) + 40
    dt = torch.bfloat16 if kv == "bf16" else torch.uint8
    kc, vc = (torch.empty((num_pages, hk, ps, D), dtype=dt, device="cuda") for _ in range(2))
    c = Prefixed(qsa, 20, [70, 9], 2, kv=kv)
    n = c.d.num_pages
    kc[-n:], vc[-n:] = c.kc, c.vc
    d = _dims(qsa, 2, c.d.max_pages, num_pages, kv, 2)
    ws = qsa.make_prefix_workspace(d, 20)
    up = num_pages - n
    for alone in (True, False):
        qsa.test_prefix_attn(d, c.q, kc, vc, c.ks, c.vs, c.args[6] + up, _up(c.args[7], up), c.args[8], c.out, ws,
                             lse=c.lse, alone=alone)
        _ok(qsa, ws)
        c.compare()


def test_prefix_refusals(qsa):
    c = Prefixed(qsa, 5, [100, 7], 2, kv="fp8").run(qsa)
    before = c.out.clone()
    d, q, kc, vc, ks, vs, xt, pt, pos, out, ws = c.args

    def call(err, match, d=d, **kw):
        a = dict(q=q, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, prefix_table=xt, page_table=pt, q_pos=pos, out=out,
                 ws=ws, lse=c.lse)
        a.update(kw)
        with pytest.raises(err, match=match):
            qsa.prefix_attn(d, **a)

    call(TypeError, "q: dtype", q=q.half())
    call(ValueError, "q: shape", q=q[:1])
    call(TypeError, "prefix_table: dtype", prefix_table=xt.long())
    call(ValueError, "prefix_table", prefix_table=xt.view(1, -1))
    call(ValueError, "prefix_table", prefix_table=None)
    call(ValueError, "CUDA", prefix_table=xt.cpu())
    call(ValueError, "contiguous", prefix_table=torch.stack([xt, xt], 1)[:, 0])
    call(qsa.QSAError, "INVALID_ARG", prefix_table=torch.zeros(d.max_pages + 1, dtype=torch.int32, device="cuda"))
    call(TypeError, "k_scale must be a tensor", k_scale=None)
    call(ValueError, "lse: shape", lse=c.lse[:, :, :8])
    call(qsa.QSAError, "WORKSPACE", ws=ws[:256])
    call(qsa.QSAError, "WORKSPACE", ws=ws[8:])
    call(ValueError, "ws must be", ws=ws.cpu())
    _ok(qsa, ws)
    assert torch.equal(out, before)
    assert qsa.prefix_workspace_size(d, 5) >= qsa.kv_workspace_size(d)
    for bad in (-1, d.max_pages + 1):
        with pytest.raises(qsa.QSAError, match="INVALID_ARG"):
            qsa.prefix_workspace_size(d, bad)


@pytest.mark.parametrize("kv,D,prefix,own,n_q,hk", [
    ("bf16", 128, 40, [5, 300, 70, 0], 4, 2), ("fp8", 128, 300, [70] * 20, 4, 2), ("fp8", 64, 9, [33, 1], 1, 4),
    ("bf16", 64, 200, [9] * 40, 2, 1), ("bf16", 256, 70, [9, 500], 2, 2), ("fp8", 256, 70, [9, 500], 2, 2)])
def test_prefix_wait_runs_out_and_reports_a_timeout(qsa, kv, D, prefix, own, n_q, hk):
    # As for the dense attention: the prefix's copies of K bring half of the
    # bytes, every CTA's wait for its first tile runs out, and all of its roles
    # end: the next calls are complete. (One row tile a CTA, two, and with an
    # E4M3 cache the warpgroup that widens; few tiles a CTA and more than the
    # copies have room for.)
    import time

    c = Prefixed(qsa, prefix, own, n_q, 16, hk, D, kv=kv)
    c.run(qsa, alone=False)
    _ok(qsa, c.ws)
    want, want_lse = c.out.clone(), c.lse.clone()
    torch.cuda.synchronize()
    t0 = time.time()
    qsa.test_prefix_attn_timeout(*c.args, lse=c.lse)
    torch.cuda.synchronize()
    waited = time.time() - t0
    st, info = qsa.check_errors(c.ws)
    assert st == qsa.ERR_TIMEOUT and info[0] == 5, info
    assert 0.2 < waited < 30, waited
    for _ in range(3):
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        c.run(qsa, alone=False)
        _ok(qsa, c.ws)
        assert torch.equal(c.out, want) and torch.equal(c.lse, want_lse)


# --------------------------------------------------------------------------
# attention weight of the cached positions
# --------------------------------------------------------------------------
class Weighed:
    def __init__(self, qsa, ctx, n_q=1, hq=16, hk=2, D=128, ps=64, kv="bf16", q_pos=None, seed=21, decay=1.0, lse=None,
                 mutate=None, sm_scale=0.0, old=None, extra_pages=0):
        B = len(ctx)
        table, num_pages = R.page_table([max(1, c) for c in ctx], ps, seed)
        self.table = torch.nn.functional.pad(table, (0, extra_pages), value=-7)
        self.kc, _, self.ks, _ = R.make_cache(num_pages, hk, ps, D, kv, seed + 1)
        self.q = _normal((B, n_q, hq, D), seed + 2)
        if q_pos is None:
            q_pos = [[max(-1, c - n_q + j) for j in range(n_q)] for c in ctx]
        self.q_pos = np.array(q_pos, dtype=np.int32)
        g = torch.Generator(device="cuda").manual_seed(seed + 3)
        cap = self.table.shape[1] * ps
        self.weight = torch.rand((B, cap), generator=g, device="cuda") if old is None else \
            torch.full((B, cap), old, device="cuda")
        self.lse = (4.0 + torch.randn((B, n_q, hq), generator=g, device="cuda")) if lse is None else lse
        if mutate:
            mutate(self)
        self.old = self.weight.clone()
        self.kv, self.B, self.decay = kv, B, decay
        self.d = _dims(qsa, B, self.table.shape[1], num_pages, kv, n_q, hq, hk, D, ps, sm_scale=sm_scale)
        self.ws = qsa.make_kv_workspace(self.d)
        self.args = (self.d, self.q, self.kc, self.ks, self.table.cuda(), _i32(self.q_pos.tolist()), self.lse, self.weight,
                     self.ws)

    def run(self, qsa, **kw):
        qsa.kv_weight(*self.args, decay=self.decay, **kw)
        return self

    def compare(self, gone=None, only=None):
        d, kc = self.d, R.f64(self.kc)
        sc = R.f64(self.ks)[None, :, None] if self.kv == "fp8" else 1.0
        scale = d.sm_scale if d.sm_scale > 0 else 1.0 / math.sqrt(d.head_dim)
        got, old, q64, lse = R.f64(self.weight), R.f64(self.old), R.f64(self.q), R.f64(self.lse)
        cap = d.max_pages * d.page_size
        for r in range(self.B):
            pos = [int(p) if 0 <= p < cap else -1 for p in self.q_pos[r]]
            top = max(pos) + 1
            assert np.array_equal(got[r, top:], old[r, top:], equal_nan=True), r
            if top == 0 or (only is not None and r not in only):
                continue
            k = R.rows(kc, self.table.numpy()[r], top) * sc
            want, tol = S.weights(q64[r], k, scale, lse[r], pos, old[r, :top], self.decay, self.kv == "fp8")
            if gone is not None and r in gone:
                at = gone[r][gone[r] < top]
                want[at], tol[at] = self.decay * old[r, at], 2.0 ** -24 * old[r, at]
            err = np.abs(got[r, :top] - want)
            assert np.all(err <= tol), (r, err.max(), (err - tol).max())
        return self


def _weight_case(qsa, *a, **kw):
    c = Weighed(qsa, *a, **kw).run(qsa)
    _ok(qsa, c.ws)
    return c.compare()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hk,D", HEADS)
@pytest.mark.parametrize("n_q", [1, 4])
def test_weight_heads(qsa, kv, hq, hk, D, n_q):
    _weight_case(qsa, [333, 70, 1, 600], n_q, hq, hk, D, 64, kv, decay=0.5)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("decay", [0.0, 0.95, 1.0])
def test_weight_lengths(qsa, kv, ps, decay):
    _weight_case(qsa, [1, 2, 15, 16, 17, 127, 128, 129, 500], 2, 8, 2, 128, ps, kv, decay=decay)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_weight_queries_anywhere(qsa, kv, D):
    pos = [[-1] * 4, [0, 1, 2, 3], [300, 3, 150, -1], [-1, 299, -1, 128], [127, 128, 129, 130], [511, 511, 511, 511]]
    _weight_case(qsa, [512] * len(pos), 4, 16, 2, D, 32, kv, q_pos=pos, decay=0.25)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ctx,n_q", [([20011], 4), ([9000, 3, 4097], 1), ([130] * 300, 1), ([40] * 700, 2)])
def test_weight_long_and_many(qsa, kv, ctx, n_q):
    _weight_case(qsa, ctx, n_q, 8, 1, 64, 16, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hk,n_q", [(1024, 1, 4), (1023, 1, 1), (256, 256, 2), (3, 1, 3)])
def test_weight_head_counts(qsa, kv, hq, hk, n_q):
    _weight_case(qsa, [200, 31], n_q, hq, hk, 64, 64, kv)


@pytest.mark.parametrize("gap", [31, 32, 33, 1000])
def test_weight_empty_requests_between(qsa, gap):
    pos = [[9, 10]] + [[-1, -1]] * gap + [[100, 101]] + [[-1, -1]] * gap
    _weight_case(qsa, [102] * len(pos), 2, 4, 1, 64, 16, "bf16", q_pos=pos)


def test_weight_without_decay_does_not_read(qsa):
    c = Weighed(qsa, [300, 9], 2, decay=0.0, old=math.nan).run(qsa)
    _ok(qsa, c.ws)
    assert torch.isfinite(c.weight[0, :300]).all() and torch.isnan(c.weight[0, 300:]).all()
    c.compare()
    c = Weighed(qsa, [300, 9], 2, decay=0.5, old=math.nan).run(qsa)
    assert torch.isnan(c.weight).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_weight_rows_left_out(qsa, kv):
    # an lse of -infinity, heads with a query that is not finite in rows that see nothing, and K behind the queries
    def poison(c):
        c.lse[0, 1, 3] = -math.inf
        c.lse[2] = -math.inf
        c.q[1, 0] = math.nan
        table = c.table.numpy()
        code = torch.tensor(math.nan).to(torch.bfloat16) if kv == "bf16" else 0x7F
        for p in (201, 210, 255):
            c.kc[int(table[0, p // 16]), :, p % 16] = code
    c = _weight_case(qsa, [256, 90, 33], 2, 16, 2, 128, 16, kv, q_pos=[[199, 200], [-1, 80], [31, 32]], mutate=poison)
    assert torch.equal(c.weight[2], c.old[2])
    # a NaN that a query does see arrives, and only there
    c = Weighed(qsa, [256], 2, 16, 2, 128, 16, kv, q_pos=[[199, 210]], mutate=lambda c: c.kc.__setitem__(
        (int(c.table[0, 205 // 16]), slice(None), 205 % 16), torch.tensor(math.nan).to(torch.bfloat16) if kv == "bf16" else 0x7F)).run(qsa)
    bad = torch.isnan(c.weight[0])
    assert bad[205] and bad.sum().item() == 1


def test_weight_of_attention_sums_to_one(qsa):
    # with the lse of the attention call, a request's new weights sum to its query rows' number
    c = Weighed(qsa, [700, 64, 3001], 4, decay=0.0)
    vc, out = torch.zeros_like(c.kc), torch.empty_like(c.q)
    qsa.paged_attn(c.d, c.q, c.kc, vc, None, None, c.args[4], c.args[5], out, c.ws, lse=c.lse)
    c.run(qsa)
    _ok(qsa, c.ws)
    for r, n in enumerate([700, 64, 3001]):
        # scores of 16 products' sums a term: both sides' errors together are below 2^-16
        assert abs(c.weight[r, :n].double().sum().item() - 64) <= 64 * 2.0 ** -16


def test_weight_reports_and_skips(qsa):
    c = Weighed(qsa, [200, 90], 2, ps=32, decay=0.5)
    t = c.args[4]
    keep = t.clone()
    for bad in (-1, c.d.num_pages):
        t[0, 3] = bad
        c.weight.copy_(c.old)
        c.run(qsa)
        st, info = qsa.check_errors(c.ws)
        assert st == qsa.ERR_BAD_INDEX and info == (2, 0, 0, bad)
        c.compare(gone={0: np.arange(96, 128)})
    t.copy_(keep)
    for bad in (-2, c.d.max_pages * 32):
        c.args[5][1, 0] = bad
        c.q_pos[1, 0] = bad
        c.weight.copy_(c.old)
        c.run(qsa)
        st, info = qsa.check_errors(c.ws)
        assert st == qsa.ERR_BAD_INDEX and info == (1, 1, 0, bad)
        c.compare()


def test_weight_same_bits_streams_and_graphs(qsa):
    c = Weighed(qsa, [700, 64, 3001, 5], 4, kv="fp8", decay=0.75).run(qsa)
    first = c.weight.clone()
    for _ in range(3):
        c.weight.copy_(c.old)
        c.run(qsa)
        assert torch.equal(c.weight, first)
    c.run(qsa)
    second = c.weight.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run(qsa)
    c.weight.copy_(c.old)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.weight, second)
    _ok(qsa, c.ws)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_weight_offsets_past_32_bits(qsa, kv):
    c = Weighed(qsa, [600, 33], 2, kv=kv)
    num_pages = (1 << 31) // (64 * 2 * 128) + 40
    kc = torch.empty((num_pages, 2, 64, 128), dtype=c.kc.dtype, device="cuda")
    n = c.d.num_pages
    kc[-n:] = c.kc
    d = _dims(qsa, 2, c.d.max_pages, num_pages, kv, 2)
    qsa.kv_weight(d, c.q, kc, c.ks, _up(c.args[4], num_pages - n), c.args[5], c.lse, c.weight, c.ws)
    _ok(qsa, c.ws)
    c.compare()


def test_weight_refusals(qsa):
    c = Weighed(qsa, [200, 90], 2, kv="fp8")
    d, q, kc, ks, pt, pos, lse, w, ws = c.args

    def call(err, match, **kw):
        a = dict(q=q, k_cache=kc, k_scale=ks, page_table=pt, q_pos=pos, lse=lse, weight=w, ws=ws)
        a.update(kw)
        with pytest.raises(err, match=match):
            qsa.kv_weight(d, **a)

    call(TypeError, "q: dtype", q=q.float())
    call(TypeError, "lse must be a tensor", lse=None)
    call(ValueError, "weight: shape", weight=w[:, :-1])
    call(TypeError, "weight: dtype", weight=w.double())
    call(TypeError, "k_scale must be a tensor", k_scale=None)
    for bad in (-0.1, 1.5, math.nan):
        call(qsa.QSAError, "INVALID_ARG", decay=bad)
    call(qsa.QSAError, "WORKSPACE", ws=ws[:128])
    call(ValueError, "ws must be", ws=None)
    _ok(qsa, ws)
    assert torch.equal(w, c.old)


@pytest.mark.parametrize("kv,hq,hk,D,n_q", [("bf16", 16, 2, 128, 4), ("fp8", 24, 8, 64, 2), ("bf16", 40, 5, 256, 4)])
def test_weight_wait_runs_out_and_reports_a_timeout(qsa, kv, hq, hk, D, n_q):
    # As for the dense attention: the hook's copies of K bring half of the bytes,
    # every CTA's wait for its first tile runs out, and all of its roles end,
    # those too that have steps ahead of them when the wait is given up (a CTA
    # has 2, 8 and 5 here): the next calls are complete.
    import time

    c = Weighed(qsa, [1500, 70, 0, 3000], n_q, hq, hk, D, kv=kv, decay=0.5).run(qsa)
    _ok(qsa, c.ws)
    want = c.weight.clone()
    torch.cuda.synchronize()
    t0 = time.time()
    qsa.test_kv_weight_timeout(*c.args, decay=c.decay)
    torch.cuda.synchronize()
    waited = time.time() - t0
    st, info = qsa.check_errors(c.ws)
    assert st == qsa.ERR_TIMEOUT and info[0] == 5, info
    assert 0.2 < waited < 30, waited
    for _ in range(3):
        c.weight.copy_(c.old)
        c.run(qsa)
        _ok(qsa, c.ws)
        assert torch.equal(c.weight, want)


# --------------------------------------------------------------------------
# eviction
# --------------------------------------------------------------------------
class Evicted:
    def __init__(self, qsa, lengths, keep, sinks=0, recent=0, hk=2, D=128, ps=64, kv="bf16", seed=31, mutate=None,
                 max_tokens=None, out_extra=0):
        B = len(lengths)
        cap = max_tokens or max(1, max(lengths))
        need = [max(1, min(max(c, 0), cap)) for c in lengths]
        table, n_in = R.page_table(need, ps, seed, spare=0)
        width = -(-cap // ps)
        self.table = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=-1)
        table_out, n_out = R.page_table([keep] * B, ps, seed + 1)
        self.table_out = torch.nn.functional.pad(table_out + n_in, (0, out_extra), value=-5)
        self.num_pages = n_in + n_out
        self.kc, self.vc, _, _ = R.make_cache(self.num_pages, hk, ps, D, kv, seed + 2)
        g = torch.Generator(device="cuda").manual_seed(seed + 3)
        self.weight = torch.exp(2 * torch.randn((B, width * ps), generator=g, device="cuda"))
        self.weight[torch.rand(self.weight.shape, generator=g, device="cuda") < 0.3] = 0
        self.lengths = list(lengths)
        self.keep, self.sinks, self.recent, self.B, self.ps = keep, sinks, recent, B, ps
        if mutate:
            mutate(self)
        self.k0, self.v0 = self.kc.clone(), self.vc.clone()
        self.d = _dims(qsa, B, width, self.num_pages, kv, 1, 2 * hk, hk, D, ps)
        self.ws = qsa.make_kv_workspace(self.d)
        self.weight_out = torch.full((B, self.table_out.shape[1] * ps), 7.0, device="cuda")
        self.kept = torch.full((B, keep), 7, dtype=torch.int32, device="cuda")
        self.new_length = torch.full((B,), 7, dtype=torch.int32, device="cuda")
        self.args = [self.d, self.kc, self.vc, self.table.cuda(), self.table_out.cuda(), _i32(self.lengths), self.weight,
                     self.weight_out, self.kept, self.new_length, self.ws]

    def run(self, qsa, **kw):
        qsa.kv_evict(*self.args, sinks=self.sinks, recent=self.recent, **kw)
        return self

    def compare(self, skip_rows=()):
        """skip_rows: (request, new position) whose K and V are not copied."""
        w = self.weight.cpu().numpy()
        bits = lambda t: t.cpu().view(torch.int16).numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()  # noqa: E731
        got, want = [bits(self.kc), bits(self.vc)], [bits(self.k0).copy(), bits(self.v0).copy()]
        src = [x.copy() for x in want]
        table, out = self.table.numpy(), self.table_out.numpy()
        for r, n in enumerate(self.lengths):
            n = n if 0 <= n <= self.weight.shape[1] else 0
            kept = S.evict(w[r], n, self.keep, self.sinks, self.recent)
            m = len(kept)
            assert int(self.new_length[r]) == m == min(n, self.keep)
            k = self.kept[r].cpu().numpy()
            assert np.array_equal(k[:m], kept) and np.all(k[m:] == -1), r
            wo = self.weight_out[r].cpu().numpy()
            assert np.array_equal(wo[:m], w[r][kept], equal_nan=True) and np.all(wo[m:] == 0), r
            to = np.array([i for i in range(m) if (r, i) not in skip_rows], dtype=int)
            for x, s in zip(want, src):
                x[out[r, to // self.ps], :, to % self.ps] = s[table[r, kept[to] // self.ps], :, kept[to] % self.ps]
        for x, y in zip(got, want):
            assert np.array_equal(x, y)
        return self


def _evict_case(qsa, *a, **kw):
    c = Evicted(qsa, *a, **kw).run(qsa)
    _ok(qsa, c.ws)
    return c.compare()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hk,D,ps", [(2, 128, 64), (1, 64, 16), (8, 256, 256), (3, 128, 32), (5, 64, 128)])
def test_evict_layouts(qsa, kv, hk, D, ps):
    _evict_case(qsa, [300, 1, 0, 97, 96, 95, 601], 96, 4, 17, hk, D, ps, kv)


@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (33, 16, 17), (500, 0, 0), (700, 3, 9),
                                               (64, 63, 0), (64, 0, 63), (64, 64, 0), (64, 0, 64)])
def test_evict_bounds(qsa, keep, sinks, recent):
    _evict_case(qsa, [500, 501, 64, 65, 2, 1, 0], keep, sinks, recent, 1, 64, 16)


@pytest.mark.parametrize("lengths,keep", [([70001], 20000), ([30000, 12, 9000], 8000), ([140] * 300, 60), ([33] * 900, 32)])
def test_evict_long_and_many(qsa, lengths, keep):
    _evict_case(qsa, lengths, keep, 4, 16, 1, 64, 16)


@pytest.mark.parametrize("lengths,keep,sinks,recent", [([30000, 12000, 7], 6000, 2000, 4000), ([30000], 64, 0, 64),
                                                       ([20001, 30000], 9000, 9000, 0)])
def test_evict_nothing_to_choose_over_several_ctas(qsa, lengths, keep, sinks, recent):
    _evict_case(qsa, lengths, keep, sinks, recent, 1, 64, 16)


@pytest.mark.parametrize("kind", ["mixed", "equal"])
def test_evict_slices_longer_than_what_is_held(qsa, kind):
    # 160 requests have a CTA each, which holds 16,384 weights of 20,000 positions
    # in shared memory; where all are equal, the last of them that stays is in front
    # of the end of those, at it and behind it
    lengths = [20000, 16384, 16385, 19999, 16400] + [0, 3, 50] * 51 + [20000, 17]
    assert len(lengths) == 160
    for keep in ((9000,) if kind == "mixed" else (16380, 16390, 17000)):
        _evict_case(qsa, lengths, keep, 4, 6, 1, 64, 16, "fp8",
                    mutate=None if kind == "mixed" else lambda c: c.weight.fill_(0.5))


@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("lengths,keep", [([30000, 9001, 40], 5000), ([700, 1001], 300)])
def test_evict_weights_at_any_offset(qsa, offset, lengths, keep):
    # arrays that start at multiples of 4 bytes, not of 16
    c = Evicted(qsa, lengths, keep, 4, 16, 1, 64, 16)
    for i in (6, 7):
        t = c.args[i]
        c.args[i] = torch.full((t.numel() + offset,), 7.0, device="cuda")[offset:].view(t.shape).copy_(t)
        assert c.args[i].data_ptr() % 16 == 4 * offset
    c.weight_out = c.args[7]
    c.run(qsa)
    _ok(qsa, c.ws)
    c.compare()


@pytest.mark.parametrize("kind", ["equal", "zeros", "special", "negative", "close", "ascending", "descending"])
def test_evict_weights(qsa, kind):
    def mutate(c):
        w = c.weight
        if kind == "equal":
            w.fill_(0.25)
        if kind == "zeros":
            w.zero_()
            w[:, ::3] = -0.0
        if kind == "special":
            w[:, ::5] = math.nan
            w[:, 1::7] = math.inf
            w[:, 2::11] = -math.inf
            w[:, 3::13] = 1e-42
            w[:, 4::17] = -1e-42
        if kind == "negative":
            w.neg_()
        if kind == "close":
            w.copy_(torch.nextafter(torch.ones_like(w), w))
            w[:, ::2] = 1.0
        if kind == "ascending":
            w.copy_(torch.arange(w.shape[1], device="cuda").float().expand_as(w))
        if kind == "descending":
            w.copy_(-torch.arange(w.shape[1], device="cuda").float().expand_as(w))
    for keep in (40, 900):
        _evict_case(qsa, [5000, 1000, 41], keep, 5, 20, 1, 64, 16, mutate=mutate)


def test_evict_only_special(qsa):
    for x in (math.nan, math.inf, -math.inf):
        _evict_case(qsa, [300], 40, 5, 20, 1, 64, 16, mutate=lambda c: c.weight.fill_(x))


def test_evict_keeps_shared_pages_where_they_are(qsa):
    # three requests over one prefix of 4 pages, in both tables, below `sinks`
    def share(c):
        c.table[:, :4] = c.table[0, :4]
        c.table_out[:, :4] = c.table[0, :4]
    c = _evict_case(qsa, [300, 151, 90], 100, 64, 8, 2, 128, 16, mutate=share)
    assert torch.equal(c.kc[c.table[0, :4].long()], c.k0[c.table[0, :4].long()])
    # a page in both tables all of whose tokens stay at their places: nothing is copied at all
    c = Evicted(qsa, [60], 100, 0, 0, 2, 128, 16, mutate=lambda c: c.table_out[:, :4].copy_(c.table[:, :4])).run(qsa)
    _ok(qsa, c.ws)
    c.compare()
    assert torch.equal(c.kc, c.k0) and torch.equal(c.vc, c.v0)


def test_evict_length_in_place_and_repeated(qsa):
    c = Evicted(qsa, [300, 20, 99], 50, 2, 10)
    c.args[9] = c.args[5]
    c.run(qsa)
    assert c.args[5].tolist() == [50, 20, 50]
    c = _evict_case(qsa, [300, 20, 99], 50, 2, 10)
    first = [x.clone() for x in (c.kc, c.vc, c.weight_out, c.kept)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run(qsa)
    for x in (c.weight_out, c.kept, c.new_length):
        x.fill_(3)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((c.kc, c.vc, c.weight_out, c.kept), first):
        assert torch.equal(x, y)
    _ok(qsa, c.ws)


def test_evict_reports_and_skips(qsa):
    c = Evicted(qsa, [-1, 300, 513, 100], 40, 2, 10, max_tokens=512)
    c.run(qsa)
    st, info = qsa.check_errors(c.ws)
    assert st == qsa.ERR_BAD_INDEX and info[0] == 8 and (info[1], info[3]) in ((0, -1), (2, 513))
    c.compare()
    for which, at, bad in (("table", 2, -1), ("table", 0, 1 << 30), ("table_out", 0, -2), ("table_out", 0, 10 ** 6)):
        c = Evicted(qsa, [300, 60], 40, 2, 10, ps=32)
        kept = S.evict(c.weight.cpu().numpy()[1], 60, 40, 2, 10) if at == 0 else S.evict(c.weight.cpu().numpy()[0], 300, 40, 2, 10)
        r = 1 if at == 0 else 0
        c.args[3 if which == "table" else 4][r, at] = bad
        c.run(qsa)
        st, info = qsa.check_errors(c.ws)
        assert st == qsa.ERR_BAD_INDEX and info == (2, r, 0, bad)
        where = kept // 32 if which == "table" else np.arange(40) // 32
        c.compare(skip_rows={(r, int(i)) for i in np.nonzero(where == at)[0]})


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_evict_offsets_past_32_bits(qsa, kv):
    c = Evicted(qsa, [600, 33], 100, 4, 10, kv=kv)
    num_pages = (1 << 31) // (64 * 2 * 128) + 40
    kc, vc = (torch.empty((num_pages, 2, 64, 128), dtype=c.kc.dtype, device="cuda") for _ in range(2))
    n = c.num_pages
    kc[-n:], vc[-n:] = c.kc, c.vc
    d = _dims(qsa, 2, c.d.max_pages, num_pages, kv, 1, 4, 2)
    up = num_pages - n
    qsa.kv_evict(d, kc, vc, _up(c.args[3], up), c.args[4] + up, *c.args[5:], sinks=4, recent=10)
    _ok(qsa, c.ws)
    c.kc, c.vc = kc[-n:].contiguous(), vc[-n:].contiguous()
    c.compare()


def test_evict_refusals(qsa):
    c = Evicted(qsa, [300, 60], 40, 2, 10)
    names = ("k_cache", "v_cache", "page_table", "page_table_out", "length", "weight", "weight_out", "kept", "new_length", "ws")
    base = dict(zip(names, c.args[1:]), sinks=2, recent=10)

    def call(err, match, **kw):
        with pytest.raises(err, match=match):
            qsa.kv_evict(c.d, **{**base, **kw})

    call(TypeError, "k_cache: dtype", k_cache=c.kc.half())
    call(ValueError, "kept must be", kept=c.kept[0])
    call(ValueError, "page_table_out must be", page_table_out=None)
    call(ValueError, "weight_out: shape", weight_out=c.weight_out[:, 1:])
    call(TypeError, "length: dtype", length=base["length"].long())
    call(qsa.QSAError, "INVALID_ARG", sinks=-1)
    call(qsa.QSAError, "INVALID_ARG", recent=-1)
    call(qsa.QSAError, "INVALID_ARG", sinks=31)
    call(qsa.QSAError, "INVALID_ARG", kept=torch.zeros((2, 65), dtype=torch.int32, device="cuda"))  # past the pages
    call(qsa.QSAError, "WORKSPACE", ws=c.ws[1:])
    same = torch.zeros((2, c.weight.shape[1]), device="cuda")
    table = torch.zeros((2, same.shape[1] // 64), dtype=torch.int32, device="cuda")
    call(qsa.QSAError, "INVALID_ARG", weight=same, weight_out=same, page_table_out=table)
    both = torch.full((2 * same.numel() - 1,), 7.0, device="cuda")  # the last element of one is the first of the other
    call(qsa.QSAError, "INVALID_ARG", weight=both[:same.numel()].view_as(same),
         weight_out=both[same.numel() - 1:].view_as(same), page_table_out=table)
    call(qsa.QSAError, "INVALID_ARG", weight_out=both[:same.numel()].view_as(same),
         weight=both[same.numel() - 1:].view_as(same), page_table_out=table)
    assert (both == 7).all()
    _ok(qsa, c.ws)
    assert (c.kept == 7).all() and (c.weight_out == 7).all()


# --------------------------------------------------------------------------
# verification of drafted tokens
# --------------------------------------------------------------------------
def _probs(shape, seed, sharp=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.softmax(sharp * torch.randn(shape, generator=g, device="cuda"), -1)


def _verify_case(qsa, target, draft, tokens, u, expect_error=None):
    B, n = tokens.shape
    ws = qsa.make_kv_workspace(qsa.make_dims(1, 1, 1, 1, 1))
    accepted = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    out = torch.full((B, n + 1), 77, dtype=torch.int32, device="cuda")
    qsa.verify_drafts(target, draft, tokens, u, accepted, out, ws)
    st, info = qsa.check_errors(ws)
    if expect_error is None:
        assert st == qsa.OK, info
    else:
        assert st == qsa.ERR_BAD_INDEX and info in expect_error
    t64, d64 = R.f64(target), None if draft is None else R.f64(draft)
    tok, uu = tokens.cpu().numpy(), u.cpu().numpy()
    for r in range(B):
        m, want = S.verify(t64[r], None if draft is None else d64[r], tok[r], uu[r])
        assert int(accepted[r]) == m, r
        assert out[r].tolist() == want, r
    return accepted, out


def _sampled(B, n, V, dt, seed, accept=0.7):
    target = _probs((B, n + 1, V), seed)
    draft = accept * target[:, :n] + (1 - accept) * target[:, :n].roll(V // 2, -1)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    tokens = torch.multinomial(draft.reshape(B * n, V), 1, generator=g).view(B, n).to(torch.int32)
    u = torch.rand((B, n + 1), generator=g, device="cuda")
    return target.to(dt), draft.to(dt), tokens, u


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (3, 2, 2), (40, 3, 31), (9, 31, 33), (20, 3, 1000), (7, 8, 4097), (2, 3, 32001),
                                   (5, 3, 100352), (2, 1, 150001), (400, 2, 257), (64, 4, 16384)])
def test_verify_sizes(qsa, dt, B, n, V):
    target, draft, tokens, u = _sampled(B, n, V, dt, 3)
    _verify_case(qsa, target, draft, tokens, u)
    _verify_case(qsa, target, None, tokens, u)


def test_verify_follows_the_plain_formula(qsa):
    # the definition in 64-bit floating point: the same tokens
    target, draft, tokens, u = _sampled(60, 3, 20011, torch.float32, 8)
    accepted, out = _verify_case(qsa, target, draft, tokens, u)
    assert set(accepted.tolist()) == {0, 1, 2, 3}
    for r in range(60):
        m = int(accepted[r])
        w = target[r, m].double()
        if m < 3:
            w = (w - draft[r, m].double()).clamp(min=0)
        c = torch.cumsum(w, 0)
        assert int(out[r, m]) == int((c <= u[r, 3].double() * c[-1]).sum())


@pytest.mark.parametrize("V", [5, 3000, 40000])
def test_verify_ragged_padded_and_bad_tokens(qsa, V):
    target, draft, tokens, u = _sampled(9, 4, V, torch.float32, 5, 0.9)
    u[:, :4] = 0  # every draft that is one is accepted
    tokens[0, 2:] = -1
    tokens[1] = -1
    tokens[2] = -2
    tokens[3, 0] = -2
    _verify_case(qsa, target, draft, tokens, u)
    # a padded request is not looked at
    target[2], draft[2], u[2] = math.nan, math.nan, math.nan
    _verify_case(qsa, target, draft, tokens, u)
    for bad in (V, -3, 2 ** 31 - 1):
        t = tokens.clone()
        t[5, 1] = bad
        t[5, 2] = V + 5  # behind the end: not looked at
        _verify_case(qsa, target, draft, t, u, expect_error=[(7, 5, 1, bad)])
    t = tokens.clone()
    t[6, 3] = -2  # only a first token of -2 stands for no request
    _verify_case(qsa, target, draft, t, u, expect_error=[(7, 6, 3, -2)])


def test_verify_random_numbers_at_the_ends(qsa):
    target, draft, tokens, u = _sampled(8, 3, 5000, torch.float32, 6)
    for x in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan, math.inf, 2.0 ** -60, 1e-45, 2.0 ** -24):
        for j in range(4):
            v = u.clone()
            v[:, j] = x
            _verify_case(qsa, target, draft, tokens, v)
        _verify_case(qsa, target, draft, tokens, torch.full_like(u, x))


def test_verify_acceptance_is_exact(qsa):
    # u q = p exactly (rejected: not below), and one step to either side
    V, n = 40, 2
    target = torch.full((6, n + 1, V), 1.0 / 64, device="cuda")
    draft = torch.full((6, n, V), 1.0 / 32, device="cuda")
    tokens = torch.full((6, n), 7, dtype=torch.int32, device="cuda")
    u = torch.full((6, n + 1), 0.5, device="cuda")
    u[1, 0] = math.nextafter(0.5, 0) if False else 0.5 - 2.0 ** -25
    u[2, 0] = 0.5 + 2.0 ** -24
    target[3, 0, 7] = float(np.nextafter(np.float32(1.0 / 64), np.float32(1)))
    draft[4, 0, 7] = float(np.nextafter(np.float32(1.0 / 32), np.float32(0)))
    # a product whose 48 bits matter: u q is below p by 2^-48 of it
    a = np.float32(1.0 - 2.0 ** -24)
    u[5, 0], draft[5, 0, 7], target[5, 0, 7] = float(a), 0.25, float(np.float32(0.25) * a)
    accepted, _ = _verify_case(qsa, target, draft, tokens, u)
    assert accepted.tolist() == [0, 1, 0, 1, 1, 0]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_verify_rows_without_weight(qsa, dt):
    V, n = 1000, 2
    target, draft, tokens, u = _sampled(6, n, V, dt, 9)
    u[:, :n] = 1.0
    draft[0] = target[0, :n]          # equal: nothing is left, the target's row as it is
    target[1] = 0                     # nothing at all: -1
    target[2, 0] = 0
    target[2, 0, 13] = 1.0            # one-hot rows, as greedy decoding has them
    draft[2, 0] = 0
    draft[2, 0, 13] = 1.0
    tokens[2, 0] = 13
    target[3, 0] = 0
    target[3, 0, V - 1] = 1.0
    tokens[3, 0] = 5
    target[4] = -target[4]            # negative counts as 0
    target[5, 0] = math.nan
    target[5, 0, 3] = 2.0             # above 1 as 1
    _verify_case(qsa, target, draft, tokens, u)
    _verify_case(qsa, target, None, tokens, u)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40000, 40001])
def test_verify_rows_without_weight_over_several_ctas(qsa, dt, V):
    # the difference is 0 everywhere: a second pass of the cluster, over the
    # target's row as it is; and rows without anything, for which y is -1
    n = 2
    target, draft, tokens, u = _sampled(5, n, V, dt, 23)
    u[:, :n] = 1.0
    draft[0], draft[1] = target[0, :n], target[1, :n]
    target[2, 0] = 0                  # nothing at all
    draft[3, 0] = 1.0                 # p is below q everywhere
    target[4, 0] = 0
    target[4, 0, V - 1] = 2.0 ** -40  # the last token alone, in the target
    draft[4, 0] = 2.0 ** -30
    for x in (0.0, 0.4, 0.9, 1.0 - 2.0 ** -24):
        u[:, n] = x
        _verify_case(qsa, target, draft, tokens, u)
    tokens[4, 0] = V - 1  # greedy, and the only token that has weight is the rejected one
    _verify_case(qsa, target, None, tokens, u)


def test_verify_tiny_probabilities(qsa):
    # sums over values from 2^-70 to 1, and a row of nothing but tiny ones
    V, n = 3001, 1
    g = torch.Generator(device="cuda").manual_seed(4)
    e = torch.randint(-70, 0, (30, n + 1, V), generator=g, device="cuda").float()
    target = torch.exp2(e) * (1 + torch.rand((30, n + 1, V), generator=g, device="cuda")) / 2 / V
    draft = target[:, :n].roll(5, -1).clone()
    tokens = torch.randint(0, V, (30, n), generator=g, device="cuda").to(torch.int32)
    u = torch.rand((30, n + 1), generator=g, device="cuda")
    target[0] = 2.0 ** -60
    target[1] = 2.0 ** -61
    target[2] = 1e-45
    _verify_case(qsa, target, draft, tokens, u)


def test_verify_differences_below_the_rounding(qsa):
    # p - q of 2^-56 everywhere, by p's and q's roundings to 2^-54 nothing: sampled
    # from p; one difference of 2^-53 among them has all the weight; values of
    # 2^-55 and below (ties go to even) none
    V, n = 2000, 1
    p = 2.0 ** -32
    target = torch.full((4, n + 1, V), p, device="cuda")
    draft = torch.full((4, n, V), p * (1 - 2.0 ** -24), device="cuda")
    tokens = torch.full((4, n), 9, dtype=torch.int32, device="cuda")
    assert (target[0, 0] > draft[0, 0]).all()
    draft[:, :, 9] = 0.5
    draft[1, 0, 1234] = p * (1 - 2.0 ** -21)
    target[2] = 2.0 ** -55
    target[3] = 2.0 ** -55
    target[3, 0, 77] = 1.5 * 2.0 ** -55
    u = torch.full((4, n + 1), 0.5, device="cuda")
    accepted, out = _verify_case(qsa, target, draft, tokens, u)
    assert accepted.tolist() == [0] * 4 and out[:, 0].tolist() == [V // 2, 1234, -1, 77]


def _heavy(dt, V, ones, rest=0.0, seed=19):
    """Two requests, a draft each: `ones` probabilities of 1, all of them a
    thread's where V is 2^20 (every 256th token of a warp's first 4,096), and
    about `rest` in all the others."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    row = torch.rand(V, generator=g, device="cuda") * (2 * rest / V)
    row[torch.arange(ones, device="cuda") * (256 if V > 4096 else 1)] = 1.0
    return row.to(dt).expand(2, 2, V).contiguous(), torch.zeros((2, 1), dtype=torch.int32, device="cuda"), g


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 1001, 1 << 20, (1 << 20) + 1])
def test_verify_rows_that_sum_to_nearly_16(qsa, dt, V):
    # sums of up to 16 less 2^-24, with the largest of them in one thread's hands
    target, tokens, g = _heavy(dt, V, 15, 0.9)
    tokens[:] = -1  # sampled from the first row
    for u in (0.0, 0.3, 0.93, 0.95, 1.0 - 2.0 ** -24):
        _verify_case(qsa, target, None, tokens, torch.full((2, 2), u, device="cuda"))
    if dt == torch.float32:
        target[:, 0] = 0
        target[:, 0, :16] = 1.0
        target[:, 0, 15] = 1.0 - 2.0 ** -24
        for u in (0.0, 0.5, 0.99, 1.0 - 2.0 ** -24):
            _verify_case(qsa, target, None, tokens, torch.full((2, 2), u, device="cuda"))
    # p of far more than 16, and p - q of 15 and a little in the same places
    target, tokens, _ = _heavy(dt, V, 15)
    draft = (torch.rand((2, 1, V), generator=g, device="cuda") / 2).to(dt)
    target[:, :1] = draft
    at = torch.arange(15, device="cuda") * (256 if V > 4096 else 1)
    target[:, 0, at], draft[:, 0, at] = 1.0, 0.0
    target[:, 0, V - 1] = draft[:, 0, V - 1] + 0.25
    tokens[:] = 20 if V <= 4096 else 21
    target[:, 0, int(tokens[0, 0])] = 0.0  # (rejected)
    for u in (0.0, 0.3, 0.95, 0.99, 1.0 - 2.0 ** -24):
        _verify_case(qsa, target, draft, tokens, torch.full((2, 2), u, device="cuda"))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,ones", [(40, 16), (40, 40), (1001, 17), (1001, 1001), (40000, 40000), (1 << 20, 16),
                                    ((1 << 20) + 1, 17), (1 << 24, 1 << 24)])
def test_verify_reports_rows_that_sum_to_16_or_more(qsa, dt, V, ones):
    # (their exact sums are past what the kernel's hold: 2^24 ones are 2^78 of its steps)
    target, tokens, _ = _heavy(dt, V, min(ones, 17))
    if ones > 17:
        target[:] = 1.0
    u = torch.full((2, 2), 0.99, device="cuda")
    ws = qsa.make_kv_workspace(qsa.make_dims(1, 1, 1, 1, 1))
    for first, row in ((-1, 0), (0, 1)):  # no draft, and one that is accepted
        tokens[:] = first
        tokens[1] = -2
        accepted = torch.full((2,), 77, dtype=torch.int32, device="cuda")
        out = torch.full((2, 2), 77, dtype=torch.int32, device="cuda")
        qsa.verify_drafts(target, None, tokens, u, accepted, out, ws)
        st, info = qsa.check_errors(ws)
        assert st == qsa.ERR_BAD_INDEX and info == (9, 0, row, 0)
        assert accepted.tolist() == [row, 0] and out.tolist() == [[0, -1] if row else [-1, -1], [-1, -1]]
    # the rows beside it are sampled from as ever
    target[1] = 0
    target[1, :, 7] = 0.5
    tokens[:] = -1
    qsa.verify_drafts(target, None, tokens, u, accepted, out, ws)
    st, info = qsa.check_errors(ws)
    assert info == (9, 0, 0, 0) and out.tolist() == [[-1, -1], [7, -1]]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_verify_strides(qsa, dt):
    B, n, V = 5, 3, 9001
    target, draft, tokens, u = _sampled(B, n, V, dt, 12)
    wide = torch.zeros((B, n + 1, V + 7), dtype=dt, device="cuda")
    for off in (0, 1, 3, 4):
        x = wide[:, :, off:off + V]
        x.copy_(target)
        _verify_case(qsa, x, draft, tokens, u)
    rows = torch.zeros((n + 1, B, V), dtype=dt, device="cuda")
    rows.copy_(target.transpose(0, 1))
    _verify_case(qsa, rows.transpose(0, 1), draft, tokens, u)
    # one distribution for all requests and rows
    _verify_case(qsa, target[:1, :1].expand(B, n + 1, V), draft[:1].expand(B, n, V), tokens, u)
    both = torch.cat([target, draft], 1)
    _verify_case(qsa, both[:, :n + 1], both[:, n + 1:], tokens, u)


def test_verify_same_result_streams_and_graphs(qsa):
    target, draft, tokens, u = _sampled(33, 3, 60001, torch.float32, 14)
    ws = qsa.make_kv_workspace(qsa.make_dims(1, 1, 1, 1, 1))
    accepted, out = _verify_case(qsa, target, draft, tokens, u)
    a2, o2 = torch.zeros_like(accepted), torch.zeros_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qsa.verify_drafts(target, draft, tokens, u, a2, o2, ws)
    for _ in range(3):
        o2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a2, accepted) and torch.equal(o2, out)
    o2.zero_()
    qsa.verify_drafts(target, draft, tokens, u, a2, o2, ws, stream=side)
    side.synchronize()
    assert torch.equal(o2, out)
    _ok(qsa, ws)


def test_verify_offsets_past_32_bits(qsa):
    V, n = 150001, 3
    B = (1 << 31) // (V * (n + 1)) + 3
    target = torch.empty((B, n + 1, V), dtype=torch.bfloat16, device="cuda")
    t, d, tokens, u = _sampled(2, n, V, torch.bfloat16, 15)
    target[-2:] = t
    all_tokens = torch.full((B, n), -2, dtype=torch.int32, device="cuda")
    all_tokens[-2:] = tokens
    uu = torch.zeros((B, n + 1), device="cuda")
    uu[-2:] = u
    ws = qsa.make_kv_workspace(qsa.make_dims(1, 1, 1, 1, 1))
    accepted = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.zeros((B, n + 1), dtype=torch.int32, device="cuda")
    qsa.verify_drafts(target, None, all_tokens, uu, accepted, out, ws)
    _ok(qsa, ws)
    a, o = _verify_case(qsa, t, None, tokens, u)
    assert torch.equal(accepted[-2:], a) and torch.equal(out[-2:], o)
    assert (out[:-2] == -1).all() and (accepted[:-2] == 0).all()


@pytest.mark.parametrize("dt,V", [(torch.float32, 3001), (torch.bfloat16, 40000)])
def test_verify_rows_that_are_not_there(qsa, dt, V):
    # Padded requests whose other tokens are in the vocabulary, and drafts that
    # end early with such tokens behind the end: through the C entry point, with
    # rows of the first requests only (what lies behind them belongs to another
    # tensor) and NaN in the rows behind the end. None of it is looked at.
    B, live, n = 6, 3, 4
    target, draft, tokens, u = _sampled(B, n, V, dt, 17, 0.9)
    u[:, :n] = 0
    tokens[live:, 0] = -2
    tokens[0, 2] = -1
    target[0, 3:], draft[0, 2:] = math.nan, math.nan
    want, want_out = _verify_case(qsa, target, draft, tokens, u)
    assert want.tolist() == [2, n, n, 0, 0, 0] and (want_out[live:] == -1).all()
    held = torch.full((2, B * (n + 1) * V), math.nan, dtype=dt, device="cuda")
    held[0, :live * (n + 1) * V] = target[:live].reshape(-1)
    held[1, :live * n * V] = draft[:live].reshape(-1)
    ws = qsa.make_kv_workspace(qsa.make_dims(1, 1, 1, 1, 1))
    accepted = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    out = torch.full((B, n + 1), 77, dtype=torch.int32, device="cuda")
    st = qsa.lib.qsa_verify_drafts(B, n, V, qsa.PROB_DTYPES[dt], held[0].data_ptr(), None, held[1].data_ptr(), None,
                                   tokens.data_ptr(), u.data_ptr(), accepted.data_ptr(), out.data_ptr(), ws.data_ptr(),
                                   ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == qsa.OK
    _ok(qsa, ws)
    assert torch.equal(accepted, want) and torch.equal(out, want_out)


def test_verify_refusals(qsa):
    target, draft, tokens, u = _sampled(4, 3, 100, torch.float32, 16)
    ws = qsa.make_kv_workspace(qsa.make_dims(1, 1, 1, 1, 1))
    base = dict(target=target, draft=draft, tokens=tokens, uniform=u,
                accepted=torch.full((4,), 7, dtype=torch.int32, device="cuda"),
                out_tokens=torch.full((4, 4), 7, dtype=torch.int32, device="cuda"), ws=ws)

    def call(err, match, **kw):
        with pytest.raises(err, match=match):
            qsa.verify_drafts(**{**base, **kw})

    call(ValueError, "target must be", target=target.half())
    call(ValueError, "target must be", target=target[0])
    call(TypeError, "draft: dtype", draft=draft.bfloat16())
    call(ValueError, "draft: shape", draft=draft[:, :2])
    call(ValueError, "last dimension", target=torch.zeros((4, 4, 200), device="cuda")[:, :, ::2])
    call(TypeError, "tokens: dtype", tokens=tokens.long())
    call(ValueError, "uniform: shape", uniform=u[:, :3])
    call(ValueError, "out_tokens: shape", out_tokens=base["out_tokens"][:, :3])
    call(ValueError, "CUDA", uniform=u.cpu())
    call(qsa.QSAError, "WORKSPACE", ws=ws[:64])
    long = torch.zeros((1, 33, 4), device="cuda")
    call(qsa.QSAError, "UNSUPPORTED", target=long, draft=None, tokens=torch.zeros((1, 32), dtype=torch.int32, device="cuda"),
         uniform=torch.zeros((1, 33), device="cuda"), accepted=base["accepted"][:1],
         out_tokens=torch.zeros((1, 33), dtype=torch.int32, device="cuda"))
    call(qsa.QSAError, "INVALID_ARG", target=target[:, :1], draft=None, tokens=tokens[:, :0], uniform=u[:, :1].contiguous(),
         out_tokens=base["out_tokens"][:, :1].contiguous())
    _ok(qsa, ws)
    assert (base["accepted"] == 7).all() and (base["out_tokens"] == 7).all()


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------
def test_calls_without_the_fast_path(qsa, monkeypatch):
    # the binding's own checks make the same calls
    c = Prefixed(qsa, 40, [70] * 20, 4, kv="fp8")
    w = Weighed(qsa, [700, 64, 3001], 4, decay=0.5)
    target, draft, tokens, u = _sampled(5, 3, 9001, torch.bfloat16, 3)
    ws = qsa.make_kv_workspace(qsa.make_dims(1, 1, 1, 1, 1))

    def everything():
        e = Evicted(qsa, [300, 20, 99], 50, 2, 10).run(qsa)
        c.run(qsa)
        w.weight.copy_(w.old)
        w.run(qsa)
        accepted, out = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros((5, 4), dtype=torch.int32, device="cuda")
        qsa.verify_drafts(target, draft, tokens, u, accepted, out, ws)
        return [x.clone() for x in (c.out, c.lse, w.weight, e.kc, e.vc, e.kept, e.weight_out, e.new_length, accepted, out)]

    fast = everything()
    assert qsa._fast is not qsa._NoFast
    monkeypatch.setattr(qsa, "_fast", qsa._NoFast)
    for a, b in zip(fast, everything()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("attend", ["prefix_attn", "test_prefix_attn"])  # (the second reads the prefix once)
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_batch_branched_from_one_context(qsa, kv, attend):
    """Three requests over a shared prefix: drafts verified, the cache's weights
    kept, the requests brought back to their bound, and decoded on from there."""
    B, n_q, hk, hq, D, ps, prefix = 3, 4, 2, 16, 128, 32, 6
    L, own = prefix * ps, [70, 33, 96]
    c = Prefixed(qsa, prefix, [n + n_q for n in own], n_q, hq, hk, D, ps, kv, seed=71, extra_pages=2)
    pages = c.d.num_pages
    keep, sinks, recent = 240, L, 16
    more = B * (-(-keep // ps) - prefix + 1)
    blank = torch.zeros((more, hk, ps, D), dtype=c.kc.dtype, device="cuda")
    kc, vc = torch.cat([c.kc, blank]), torch.cat([c.vc, blank])
    d = _dims(qsa, B, c.d.max_pages, pages + more, kv, n_q, hq, hk, D, ps)
    ws = qsa.make_prefix_workspace(d, prefix)
    table, shared = c.full.cuda(), c.args[6]
    rope = qsa.make_rope(D)
    k, v, q = _normal((B, n_q, hk, D), 72), _normal((B, n_q, hk, D), 73), _normal((B, n_q, hq, D), 74)
    pos = _i32([[L + n + j for j in range(n_q)] for n in own])
    q_rot, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((B, n_q, hq), device="cuda")
    qsa.kv_append(d, k, v, kc, vc, c.ks, c.vs, table, pos, ws, rope=rope, q=q, q_out=q_rot)
    getattr(qsa, attend)(d, q_rot, kc, vc, c.ks, c.vs, shared, table, pos, out, ws, lse=lse)
    weight = torch.zeros((B, d.max_pages * ps), device="cuda")
    qsa.kv_weight(d, q_rot, kc, c.ks, table, pos, lse, weight, ws)
    # the model's head stands outside; its probabilities are given
    V = 501
    target, draft, tokens, u = _sampled(B, n_q - 1, V, torch.float32, 75, 0.9)
    u[1, 0] = 0.999
    accepted = torch.empty(B, dtype=torch.int32, device="cuda")
    out_tokens = torch.empty((B, n_q), dtype=torch.int32, device="cuda")
    qsa.verify_drafts(target, draft, tokens, u, accepted, out_tokens, ws)
    length = (pos[:, 0] + 1 + accepted).to(torch.int32)  # rejected drafts' slots are behind it
    table_out = torch.full((B, 10), -1, dtype=torch.int32, device="cuda")
    table_out[:, :prefix] = shared
    table_out[:, prefix:prefix + 2] = _i32([[pages + 2 * r, pages + 2 * r + 1] for r in range(B)])
    weight_out, kept = torch.empty((B, 10 * ps), device="cuda"), torch.empty((B, keep), dtype=torch.int32, device="cuda")
    new_length = torch.empty_like(length)
    qsa.kv_evict(d, kc, vc, table, table_out, length, weight, weight_out, kept, new_length, ws, sinks=sinks, recent=recent)
    d1 = _dims(qsa, B, 10, pages + more, kv, 1, hq, hk, D, ps)
    ws1 = qsa.make_prefix_workspace(d1, prefix)
    q1 = _normal((B, 1, hq, D), 76)
    out1, lse1 = torch.empty_like(q1), torch.empty((B, 1, hq), device="cuda")
    last = (new_length - 1).view(B, 1).contiguous()
    getattr(qsa, attend)(d1, q1, kc, vc, c.ks, c.vs, shared, table_out, last, out1, ws1, lse=lse1)
    _ok(qsa, ws)
    _ok(qsa, ws1)

    # the same in 64 bits
    sc = [R.f64(s)[None, :, None] if kv == "fp8" else 1.0 for s in (c.ks, c.vs)]
    for r in range(B):
        top = L + own[r] + n_q
        kk, vv = (R.rows(R.f64(x), c.full.numpy()[r], top) * s for x, s in zip((kc, vc), sc))
        for j in range(n_q):
            ref, rl, mag, qk, small = R.attention(R.f64(q_rot)[r, j], kk, vv, 1 / math.sqrt(D), 0, L + own[r] + j + 1)
            tol, tol_l = S.attn_tol(ref, mag, rl, qk, D, kv, small)
            assert np.all(np.abs(R.f64(out)[r, j] - ref) <= tol) and np.all(np.abs(R.f64(lse)[r, j] - rl) <= tol_l)
        want, tol = S.weights(R.f64(q_rot)[r], kk, 1 / math.sqrt(D), R.f64(lse)[r], pos[r].tolist(), np.zeros(top), 1.0, kv == "fp8")
        assert np.all(np.abs(R.f64(weight)[r, :top] - want) <= tol)
        m, toks = S.verify(R.f64(target)[r], R.f64(draft)[r], tokens[r].tolist(), u[r].tolist())
        assert int(accepted[r]) == m and out_tokens[r].tolist() == toks
        n = L + own[r] + 1 + m
        stay = S.evict(weight[r].cpu().numpy(), n, keep, sinks, recent)
        assert kept[r, :len(stay)].tolist() == stay.tolist() and int(new_length[r]) == len(stay)
        ref, rl, mag, qk, small = R.attention(R.f64(q1)[r, 0], kk[stay], vv[stay], 1 / math.sqrt(D), 0, len(stay))
        tol, tol_l = S.attn_tol(ref, mag, rl, qk, D, kv, small)
        assert np.all(np.abs(R.f64(out1)[r, 0] - ref) <= tol) and np.all(np.abs(R.f64(lse1)[r, 0] - rl) <= tol_l)
    assert torch.equal(kc[shared.long()], c.kc[shared.long()])  # the prefix was not touched


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_decoding_on_after_an_eviction(qsa, kv):
    """Requests decoded on from a bounded cache as qsa_serve.h says: tokens
    rotated at their true positions and appended at their places, the weights
    taken of the tokens that verification keeps; evicted again."""
    B, n_q, hk, hq, D, ps, keep, sinks, recent = 3, 3, 2, 8, 64, 16, 64, 4, 16
    lengths = [150, 97, 33]
    rope, top = qsa.make_rope(D), max(lengths)
    table, pages = R.page_table(lengths, ps, 81, spare=0)
    width, more = -(-(keep + 2 * n_q) // ps), 2 * B * -(-(keep + 2 * n_q) // ps)
    kc, vc, ks, vs = R.make_cache(pages + more, hk, ps, D, kv, 82)
    tables = [table] + [(torch.arange(B * width, dtype=torch.int32) + pages + i * B * width).view(B, width) for i in range(2)]
    d = _dims(qsa, B, table.shape[1], pages + more, kv, n_q, hq, hk, D, ps)
    d1 = _dims(qsa, B, width, pages + more, kv, n_q, hq, hk, D, ps)
    ws = qsa.make_kv_workspace(d)
    k, v = _normal((B, top, hk, D), 83), _normal((B, top, hk, D), 84)
    pos = torch.arange(top, dtype=torch.int32).expand(B, -1).clone()
    for r, n in enumerate(lengths):
        pos[r, n:] = -1
    qsa.kv_append(d, k, v, kc, vc, ks, vs, table.cuda(), pos.cuda(), ws, rope=rope)
    w, amp = R.frequencies(D)
    key_of = [list(R.rotate(R.f64(k)[r, :n], np.arange(n), w, amp, "half")) for r, n in enumerate(lengths)]
    value_of = [list(R.f64(v)[r, :n]) for r, n in enumerate(lengths)]
    true = [list(range(n)) for n in lengths]  # of the token at each place
    had = list(lengths)
    g = torch.Generator(device="cuda").manual_seed(85)
    weight = torch.rand((B, table.shape[1] * ps), generator=g, device="cuda")
    weight[pos_behind(lengths, weight.shape[1])] = 0
    length = _i32(lengths)
    now, dims = tables[0], d
    for step, (after, accepted) in enumerate(zip(tables[1:], ([2, 0, 1], [1, 2, 0]))):
        # bounded again
        out_w = torch.empty((B, width * ps), device="cuda")
        kept, place = torch.empty((B, keep), dtype=torch.int32, device="cuda"), torch.empty_like(length)
        qsa.kv_evict(dims, kc, vc, now.cuda(), after.cuda(), length, weight, out_w, kept, place, ws, sinks=sinks, recent=recent)
        for r in range(B):
            stay = S.evict(weight[r].cpu().numpy(), int(length[r]), keep, sinks, recent)
            assert kept[r, :len(stay)].tolist() == stay.tolist()
            true[r] = [true[r][i] for i in stay]
        now, dims, weight, length = after, d1, out_w, place.clone()
        assert any(int(length[r]) < had[r] for r in range(B))
        # n_q tokens more: rotated where they truly are, appended where there is room
        q, k, v = (_normal((B, n_q, h, D), 90 + 3 * step + i) for i, h in enumerate((hq, hk, hk)))
        j = torch.arange(n_q, device="cuda")
        at, true_at = ((x.view(B, 1) + j).to(torch.int32) for x in (length, _i32(had)))
        q_rot, k_rot = torch.empty_like(q), torch.empty_like(k)
        qsa.rope(rope, q, true_at, q_rot)
        qsa.rope(rope, k, true_at, k_rot)
        qsa.kv_append(d1, k_rot, v, kc, vc, ks, vs, now.cuda(), at, ws)
        out, lse = torch.empty_like(q), torch.empty((B, n_q, hq), device="cuda")
        qsa.paged_attn(d1, q_rot, kc, vc, ks, vs, now.cuda(), at, out, ws, lse=lse)
        m = _i32(accepted)
        seen = torch.where(j <= m.view(B, 1), at, -1).to(torch.int32)
        old = weight.clone()
        qsa.kv_weight(d1, q_rot, kc, ks, now.cuda(), seen, lse, weight, ws, decay=0.5)
        _ok(qsa, ws)
        sc = [R.f64(s)[None, :, None] if kv == "fp8" else 1.0 for s in (ks, vs)]
        for r in range(B):
            n = int(length[r])
            key_of[r] += list(R.rotate(R.f64(k)[r], np.arange(had[r], had[r] + n_q), w, amp, "half"))
            value_of[r] += list(R.f64(v)[r])
            true[r] += list(range(had[r], had[r] + n_q))
            kk, vv = (R.rows(R.f64(x), now.numpy()[r], n + n_q) * s for x, s in zip((kc, vc), sc))
            # the cache holds the tokens at their true positions: a key is rounded to
            # BF16 and, with E4M3, to half a step of its code (2^-10 of the scale next
            # to 0); the rotation's own arithmetic is FP32
            for have, want in ((kk, key_of), (vv, value_of)):
                want = np.array([want[r][t] for t in true[r]])
                tol = (2.0 ** -8 + 2.0 ** -20) * np.abs(want) + 2.0 ** -20 * np.abs(want).max(-1, keepdims=True)
                if kv == "fp8":
                    tol = tol + 2.0 ** -4 * (np.abs(want) + tol) + 2.0 ** -10 * (sc[0] if have is kk else sc[1])
                assert np.all(np.abs(have - want) <= tol)
            for i in range(n_q):
                ref, rl, mag, qk, small = R.attention(R.f64(q_rot)[r, i], kk, vv, 1 / math.sqrt(D), 0, n + i + 1)
                tol, tol_l = S.attn_tol(ref, mag, rl, qk, D, kv, small)
                assert np.all(np.abs(R.f64(out)[r, i] - ref) <= tol) and np.all(np.abs(R.f64(lse)[r, i] - rl) <= tol_l)
            # rejected drafts: no weight from them, none at their places
            top = n + accepted[r] + 1
            want, tol = S.weights(R.f64(q_rot)[r], kk[:top], 1 / math.sqrt(D), R.f64(lse)[r], seen[r].tolist(),
                                  R.f64(old)[r, :top], 0.5, kv == "fp8")
            assert np.all(np.abs(R.f64(weight)[r, :top] - want) <= tol) and (weight[r, top:] == 0).all()
            true[r] = true[r][:top]
            had[r] += accepted[r] + 1
            key_of[r], value_of[r] = key_of[r][:had[r]], value_of[r][:had[r]]
        length = (length + m + 1).to(torch.int32)


def pos_behind(lengths, n):
    return torch.arange(n, device="cuda").view(1, -1) >= _i32(lengths).view(-1, 1)


def test_sparse_step_after_an_eviction(qsa):
    """The sparse step on an evicted cache, its compressed keys made anew from the
    index keys in their new order, against the oracle on the tokens that stay."""
    from block_sparse_attention_qsa_gb300 import synth
    from oracle import qsa_oracle as O

    B, n_q, keep, sinks, recent = 2, 4, 2500, 4, 100
    spec = synth.Spec("evicted", B, n_q, [3000, 2700], 1, "bf16", True, 4243)
    inp = {k: v.cuda() for k, v in synth.make_inputs(spec).items()}
    d = qsa.dims_for_spec(spec)
    ps, pages = d.page_size, inp["k_cache"].shape[0]
    width = -(-keep // ps)
    blank = torch.zeros((B * width, *inp["k_cache"].shape[1:]), dtype=torch.bfloat16, device="cuda")
    kc, vc = torch.cat([inp["k_cache"], blank]), torch.cat([inp["v_cache"], blank])
    k0, v0 = kc.clone(), vc.clone()
    table_out = (torch.arange(B * width, dtype=torch.int32, device="cuda") + pages).view(B, width)
    length = inp["q_pos"].amax(1) + 1
    g = torch.Generator(device="cuda").manual_seed(91)
    weight = torch.rand((B, d.max_pages * ps), generator=g, device="cuda")
    weight_out, kept = torch.empty((B, width * ps), device="cuda"), torch.empty((B, keep), dtype=torch.int32, device="cuda")
    d_all = _dims(qsa, B, d.max_pages, pages + B * width, "bf16", n_q, 16, 2, 128, ps)
    new_length = torch.empty_like(length)
    ws = qsa.make_kv_workspace(d_all)
    qsa.kv_evict(d_all, kc, vc, inp["page_table"], table_out, length, weight, weight_out, kept, new_length, ws,
                 sinks=sinks, recent=recent)
    _ok(qsa, ws)
    assert new_length.tolist() == [keep] * B
    # the newest n_q tokens are the verify queries', at the end of either order
    q_pos = (new_length.view(B, 1) - n_q + torch.arange(n_q, device="cuda")).to(torch.int32)
    order = kept.long()
    idx = torch.stack([inp["idx_keys"][r][order[r]] for r in range(B)]).contiguous()
    blocks = keep // 4
    d1 = qsa.make_dims(B, n_q, blocks, width, pages + B * width, 1, "bf16", ps)
    comp = torch.zeros((B, blocks, 1, 128), dtype=torch.bfloat16, device="cuda")
    ws1 = qsa.make_workspace(d1)
    qsa.compress_keys(d1, idx, q_pos, comp, ws1)
    out = torch.empty((B, n_q, 16, 128), dtype=torch.bfloat16, device="cuda")
    sel = torch.empty((B, n_q, 2051), dtype=torch.int32, device="cuda")
    qsa.decode(d1, inp["q_idx"], comp, inp["q"], kc, vc, inp["k_scale"], inp["v_scale"], table_out, q_pos, out, ws1,
               sel_pos=sel)
    _ok(qsa, ws1)
    # the oracle: a cache in which the tokens that stay lie in their order, taken from the cache before the call
    bits = lambda t: t.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    at = torch.arange(keep, device="cuda")
    for r in range(B):
        page = inp["page_table"][r].long()[order[r] // ps]
        for x in (k0, v0):
            x[table_out[r].long()[at // ps], :, at % ps] = x[page, :, order[r] % ps]
    npi = {"q_idx": bits(inp["q_idx"]), "q": bits(inp["q"]), "k_cache": bits(k0), "v_cache": bits(v0),
           "page_table": table_out.cpu().numpy(), "q_pos": q_pos.cpu().numpy(),
           "kc": np.stack([O.compress_keys(bits(idx[r]), blocks) for r in range(B)])}
    ref = O.decode_step(npi, "bf16")
    for (r, j), o in ref["out"].items():
        assert np.array_equal(sel[r, j].cpu().numpy(), ref["sel_pos"][(r, j)])
        assert np.max(np.abs(out[r, j].float().cpu().numpy() - o)) <= 1e-2
