"""The operators round the paged cache on the GPU against 64-bit references.

Tolerances. BF16 values are off by at most 2^-8 of themselves (half a step),
E4M3 codes by 2^-4 of themselves, or 2^-10 below the normal range. Rotation: a
pair's products and sincospi carry FP32 errors of a few 2^-24 of |x_a| + |x_b|;
2^-20 of it is allowed. Attention: see _attn_tol.
"""

import math

import numpy as np
import pytest
import torch

from tests import _kv_ref as R

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
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


def _i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def _dims(qsa, B, max_pages, num_pages, kv="bf16", n_q=1, hq=16, hk=2, D=128, ps=64, **kw):
    return qsa.make_dims(B, n_q, max(1, max_pages * ps // 4), max_pages, num_pages, 1, kv, ps, hq, hk, D, **kw)


# --------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------
SCALINGS = [dict(), dict(base=1e6, scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
            dict(scaling="yarn", factor=16.0, orig_len=4096.0)]


def _check_rotation(got, x, pos, w, amp, layout, inverse=False):
    x64 = R.f64(x)
    ref = R.rotate(x64, pos, w, amp, layout, inverse)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * amp * R.pair_size(x64, w, layout)
    err = np.abs(R.f64(got) - ref)
    assert np.all(err <= tol), (err - tol).max()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (256, 256), (128, 32), (128, 2), (256, 66), (64, 10), (128, 72)])
@pytest.mark.parametrize("kw", SCALINGS, ids=lambda k: k.get("scaling", "none"))
def test_rope(qsa, layout, D, rot, kw):
    if rot == 2 and kw.get("scaling") == "ntk":
        pytest.skip("no NTK base for one pair")
    B, n, H = 2, 7, 3
    x = _normal((B, n, H, D), rot + D)
    pos = np.array([[0, 1, 2, 63, 4095, 131071, 1048575], [5, -1, 2 ** 31 - 1, 1000003, -1, 77, 12]])
    rope = qsa.make_rope(rot, layout=layout, **kw)
    w, amp = R.frequencies(rot, **kw)
    for inverse in (False, True):
        y = torch.full_like(x, 7.0)
        qsa.rope(rope, x, _i32(pos), y, inverse=inverse)
        live = pos >= 0
        xs, ys = x.cpu()[torch.from_numpy(live)], y.cpu()[torch.from_numpy(live)]
        _check_rotation(ys, xs, pos[live], w, amp, layout, inverse)
        assert torch.all(y.cpu()[torch.from_numpy(~live)] == 7.0)  # no token: left as it was
        # from component rot on: the same bits
        assert torch.equal(ys[..., rot:], xs[..., rot:])
    z = x.clone()
    qsa.rope(rope, z, _i32(pos), z, inverse=True)  # in place
    assert torch.equal(z[torch.from_numpy(live).cuda()], y[torch.from_numpy(live).cuda()])


@pytest.mark.parametrize("n", [1, 3, 4, 5, 700])
@pytest.mark.parametrize("H", [1, 16, 65])
def test_rope_sizes(qsa, n, H):
    x = _normal((3, n, H, 128), n + H)
    pos = np.arange(3)[:, None] * 1000 + np.arange(n)
    rope = qsa.make_rope(64)
    y = torch.empty_like(x)
    qsa.rope(rope, x, _i32(pos), y)
    w, amp = R.frequencies(64)
    _check_rotation(y, x, pos, w, amp, "half")


def test_rope_strides(qsa):
    # heads of a packed projection, tokens and heads in another order, an odd
    # row start, a broadcast batch: all the same values as contiguous copies
    B, n, H, D = 2, 5, 4, 64
    pos = _i32(np.arange(B * n).reshape(B, n) * 37)
    rope = qsa.make_rope(64)
    views = {
        "packed": _normal((B, n, H + 3, D), 1)[:, :, 2:2 + H],
        "heads first": _normal((B, H, n, D), 2).transpose(1, 2),
        "tokens first": _normal((n, B, H, D), 3).transpose(0, 1),
        "odd start": _normal((B, n, H, D + 1), 4)[..., 1:],
        "broadcast": _normal((1, n, H, D), 5).expand(B, n, H, D),
        "one head for all": _normal((B, n, 1, D), 6).expand(B, n, H, D),
    }
    for name, x in views.items():
        want, got = torch.empty((B, n, H, D), dtype=torch.bfloat16, device="cuda"), None
        qsa.rope(rope, x.contiguous(), pos, want)
        got = torch.empty_like(want)
        qsa.rope(rope, x, pos, got)
        assert torch.equal(want, got), name
        buf = torch.full((B, n, H + 1, D + 1), 3.0, dtype=torch.bfloat16, device="cuda")
        out = buf[:, :, 1:, :D]
        qsa.rope(rope, x, pos, out)
        assert torch.equal(want, out), name
        assert torch.all(buf[:, :, 0] == 3.0) and torch.all(buf[..., D] == 3.0), name
    packed = views["packed"]
    want = torch.empty((B, n, H, D), dtype=torch.bfloat16, device="cuda")
    qsa.rope(rope, packed.contiguous(), pos, want)
    qsa.rope(rope, packed, pos, packed)
    assert torch.equal(want, packed)


def test_rope_strides_of_single_elements(qsa):
    # a dimension of one element has no stride: in place through another view
    # of the same rows, and an odd stride of it does not matter
    x = _normal((1, 1, 4, 64), 7)
    want, rope, pos = torch.empty_like(x), qsa.make_rope(64), _i32([[1234]])
    qsa.rope(rope, x, pos, want)
    qsa.rope(rope, x.as_strided(x.shape, (9, 7, 64, 1)), pos, x.as_strided(x.shape, (1, 256, 64, 1)))
    assert torch.equal(x, want)


def test_rope_gradient(qsa):
    # inverse is the gradient: the transpose of the forward matrix (formula),
    # and <dy, rope(x + h e) - rope(x - h e)> / 2h (differences)
    B, n, H, D, rot = 1, 3, 2, 64, 32
    kw = dict(scaling="yarn", factor=16.0, orig_len=64.0)
    rope = qsa.make_rope(rot, layout="interleaved", **kw)
    w, amp = R.frequencies(rot, **kw)
    pos = np.array([[3, 500, 100000]])
    x, dy = _normal((B, n, H, D), 11), _normal((B, n, H, D), 12)
    dx = torch.empty_like(dy)
    qsa.rope(rope, dy, _i32(pos), dx, inverse=True)
    _check_rotation(dx, dy, pos, w, amp, "interleaved", inverse=True)
    x64, dy64, dx64 = R.f64(x), R.f64(dy), R.f64(dx)
    # the forward map is linear, so a step of 1 has no truncation error
    for at in [(0, 0, 0, 0), (0, 1, 1, 7), (0, 2, 0, 30), (0, 2, 1, 31), (0, 1, 0, 40)]:
        e = np.zeros_like(x64)
        e[at] = 1.0
        diff = (R.rotate(x64 + e, pos, w, amp, "interleaved") - R.rotate(x64 - e, pos, w, amp, "interleaved")) / 2
        want = float((dy64 * diff).sum())
        assert abs(dx64[at] - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -20 * 4


# --------------------------------------------------------------------------
# cache write
# --------------------------------------------------------------------------
def _positions(starts, lengths, n):
    pos = np.full((len(starts), n), -1, dtype=np.int32)
    for r, (s, m) in enumerate(zip(starts, lengths)):
        pos[r, :m] = np.arange(s, s + m)
    return pos


APPENDS = [
    # starts, lengths, n, hq, hk, D, page_size
    ([0], [1], 1, 16, 2, 128, 64),
    ([62, 0, 127], [4, 0, 3], 4, 16, 2, 128, 64),
    ([5, 1000], [33, 17], 33, 3, 1, 64, 16),
    ([250, 3], [9, 9], 9, 4, 4, 256, 256),
    ([1], [701], 701, 8, 8, 128, 32),
    ([7, 7, 7, 7, 7], [2, 1, 2, 0, 2], 2, 64, 1, 128, 128),
    ([15, 0], [3, 2], 3, 1024, 128, 64, 16),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"n{c[2]}-{c[3]}/{c[4]}-d{c[5]}-p{c[6]}")
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("rot,layout", [(0, "half"), (1, "half"), (1, "interleaved"), (6, "half"), (6, "interleaved")])
@pytest.mark.parametrize("packed", [False, True, "odd"])  # odd: rows that cannot be read 16 bytes at a time
def test_append(qsa, case, kv, rot, layout, packed):
    starts, lengths, n, hq, hk, D, ps = case
    rot = {0: 0, 1: D}.get(rot, rot)  # none, all of the head, three pairs
    B = len(starts)
    pos = _positions(starts, lengths, n)
    table, num_pages = R.page_table([s + m for s, m in zip(starts, lengths)], ps, 3)
    kc, vc, ks, vs = R.make_cache(num_pages, hk, ps, D, kv, 21)
    before = [f.clone() for f in (kc, vc)]
    qkv = _normal((B, n, hq + 2 * hk, D + (packed == "odd")), 22)[..., :D]
    qkv[0, 0, hq, 0] = 1e4  # past the largest code: clamped
    q, k, v = (qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:])
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    d = _dims(qsa, B, table.shape[1], num_pages, kv, hq=hq, hk=hk, D=D, ps=ps)
    ws = qsa.make_kv_workspace(d)
    rope = qsa.make_rope(rot, layout=layout) if rot else None
    q_out = torch.full((B, n, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    extra = dict(rope=rope, q=q, q_out=q_out) if rope else {}
    qsa.kv_append(d, k, v, kc, vc, ks, vs, table.cuda(), _i32(pos), ws, **extra)
    _ok(qsa, ws)
    w, amp = R.frequencies(rot) if rot else (np.zeros(0), 1.0)
    live = torch.from_numpy(pos >= 0)
    if rope:
        _check_rotation(q_out.cpu()[live], q.cpu()[live], pos[pos >= 0], w, amp, layout)
        assert torch.all(q_out.cpu()[~live] == 7.0)
    table = table.numpy()
    sk, sv = R.f64(ks)[:, None], R.f64(vs)[:, None]
    touched = np.zeros((num_pages, ps), dtype=bool)
    got = [R.f64(kc), R.f64(vc)]
    for r in range(B):
        p = pos[r, :lengths[r]]
        page, slot = table[r, p // ps], p % ps
        touched[page, slot] = True
        k64, v64 = R.f64(k[r, :lengths[r]]), R.f64(v[r, :lengths[r]])
        rk = R.rotate(k64, p, w, amp, layout)
        slack = 2.0 ** -20 * R.pair_size(k64, w, layout)
        gk, gv = got[0][page, :, slot], got[1][page, :, slot]
        if kv == "bf16":
            assert np.all(np.abs(gk - rk) <= 2.0 ** -8 * np.abs(rk) + slack)
            assert np.array_equal(gv, v64)
        else:
            z = np.clip(rk / sk, -448, 448)
            # half a step of the code, and FP32's division on top (2^-24, far inside the slack)
            assert np.all(np.abs(gk - z) <= 2.0 ** -4 * np.abs(z) + 2.0 ** -10 + slack / sk + 2.0 ** -22 * np.abs(z))
            want = (v[r, :lengths[r]].float() / vs.view(1, -1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
            assert np.array_equal(gv, want.float().cpu().numpy().astype(np.float64))
    for c, b in zip((kc, vc), before):  # every other slot as it was
        other = torch.from_numpy(~touched).cuda()
        assert torch.equal(c.transpose(1, 2)[other], b.transpose(1, 2)[other])


@pytest.mark.parametrize("odd", [False, True])
def test_append_every_value_by_every_scale(qsa, odd):
    # every BF16 value by scales of all sizes: the codes of the FP32 quotient
    # (odd: rows that cannot be read 16 bytes at a time)
    scales = np.array([1.0, 0.013, 3.7e-5, 2.0 ** -61, 2.0 ** 75, -0.3, 1 / 448, 5.9e17, 3e38, 1e-41, 0.0, -1.7e-6,
                       math.inf, 2.0 ** -60, 2.0 ** 60, 1.9999999], dtype=np.float32)
    hk, D, ps, n = len(scales), 128, 64, 512
    d = _dims(qsa, 1, n // ps, n // ps, "fp8", 1, hk, hk, D, ps)
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(1, n, 1, D)
    buf = torch.zeros((1, n, hk, D + 1), dtype=torch.bfloat16)
    buf[..., :D] = x
    k = buf.cuda()[..., :D] if odd else x.expand(1, n, hk, D).contiguous().cuda()
    kc, vc = (torch.zeros((n // ps, hk, ps, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    sc, ws = torch.from_numpy(scales).cuda(), qsa.make_kv_workspace(d)
    pt, pos = _i32([np.arange(n // ps)]), _i32([np.arange(n)])
    qsa.kv_append(d, k, k, kc, vc, sc, sc, pt, pos, ws)
    with np.errstate(all="ignore"):
        quot = x.float().numpy()[0] / scales[None, :, None]  # [n][hk][D], FP32
    lim = torch.from_numpy(np.clip(quot, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    want = lim.view(n // ps, ps, hk, D).transpose(1, 2).contiguous()
    for got in (kc.cpu(), vc.cpu()):
        nan = (want & 0x7f) == 0x7f
        assert torch.equal((got & 0x7f)[nan], want[nan] & 0x7f)
        assert torch.equal(got[~nan], want[~nan])
    _ok(qsa, ws)


def test_append_special_values(qsa):
    # E4M3: NaN stays NaN, infinities and large values clamp, ties go to even,
    # the range below the normals; BF16: every bit pattern is kept
    d = _dims(qsa, 1, 1, 1, "fp8", hq=1, hk=1, D=64)
    ws = qsa.make_kv_workspace(d)
    vals = [math.nan, math.inf, -math.inf, 448.0, 464.0, 465.0, 1e30, -1e30, 0.0, -0.0, 2.0 ** -9, 2.0 ** -10,
            3 * 2.0 ** -10, 2.0 ** -11, 17.0, 18.0, 19.0, 25.0, 27.0, -17.0, 1.0625, 1.1875, 2.0 ** -6, 2.0 ** -7]
    x = torch.zeros(1, 1, 1, 64)
    x[0, 0, 0, :len(vals)] = torch.tensor(vals)
    x = x.to(torch.bfloat16).cuda()
    kc, vc = (torch.full((1, 1, 64, 64), 0x33, dtype=torch.uint8, device="cuda") for _ in range(2))
    one = torch.ones(1, device="cuda")
    qsa.kv_append(d, x, x, kc, vc, one, one, _i32([[0]]), _i32([[9]]), ws)
    _ok(qsa, ws)
    f = x.float().cpu().view(-1)
    want = torch.where(f.isnan(), f, f.clamp(-448, 448)).to(torch.float8_e4m3fn).float()
    for c in (kc, vc):
        got = c.cpu().view(torch.float8_e4m3fn)[0, 0, 9].float()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(), want.nan_to_num())
        assert torch.equal(torch.signbit(got[~got.isnan()]), torch.signbit(want[~want.isnan()]))
        rest = torch.ones(64, dtype=torch.bool)
        rest[9] = False
        assert torch.all(c.cpu()[0, 0, rest] == 0x33)
    bits = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int16).view(1, 512, 2, 64).view(torch.bfloat16).cuda()
    d = _dims(qsa, 1, 8, 8, "bf16", hq=2, hk=2, D=64)
    kc, vc = (torch.zeros((8, 2, 64, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = qsa.make_kv_workspace(d)
    pos = _i32(np.arange(512)[None])
    qsa.kv_append(d, bits, bits, kc, vc, None, None, _i32([np.arange(8)]), pos, ws)
    ko, vo = torch.empty_like(bits), torch.empty_like(bits)
    qsa.kv_gather(d, kc, vc, None, None, _i32([np.arange(8)]), pos, ko, vo, ws)
    _ok(qsa, ws)
    nan = bits.isnan()
    for o in (ko, vo):
        assert torch.equal(o.view(torch.int16)[~nan], bits.view(torch.int16)[~nan]) and torch.all(o[nan].isnan())


def test_append_reports_and_skips(qsa):
    ps, B, n = 16, 4, 3
    table = np.array([[0, 1], [2, 3], [4, 99], [6, 7]], dtype=np.int32)
    kc, vc, ks, vs = R.make_cache(8, 2, ps, 64, "bf16", 5)
    x = _normal((B, n, 4, 64), 6)
    d = _dims(qsa, B, 2, 8, "bf16", hq=2, hk=2, D=64, ps=ps)
    ws = qsa.make_kv_workspace(d)
    rope = qsa.make_rope(64)
    cases = [
        # positions, (kind, request, token, value) of one of the faults (None: not the only one), skipped
        # (request, token)s; K and V only for kind 2
        ([[0, 1, 2], [4, 6, 5], [0, 1, 2], [0, 1, 2]], (6, 1, None, None), [(1, 1), (1, 2)]),
        ([[30, 31, 32], [4, 5, 6], [0, 1, 2], [0, 1, 2]], (1, 0, 2, 32), [(0, 2)]),
        ([[0, 1, -2], [4, 5, 6], [0, 1, 2], [0, 1, 2]], (1, 0, 2, -2), [(0, 2)]),
        ([[0, 1, 2], [4, 5, 6], [15, 16, 17], [0, 1, 2]], (2, 2, None, 99), [(2, 1), (2, 2)]),
        ([[0, 1, 2], [-1, 5, 6], [0, -1, 2], [0, 1, 2]], (6, 1, None, None), [(1, 0), (1, 1), (1, 2), (2, 1)]),
    ]
    for pos, want, skipped in cases:
        kc.fill_(9.0), vc.fill_(9.0)
        q_out = torch.full((B, n, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        qsa.kv_append(d, x[:, :, :2], x[:, :, 2:], kc, vc, None, None, _i32(table), _i32(pos), ws, rope=rope,
                      q=x[:, :, :2], q_out=q_out)
        st, info = qsa.check_errors(ws)
        assert st == qsa.ERR_BAD_INDEX
        assert all(b is None or a == b for a, b in zip(info, want)), (info, want)
        written = np.zeros((8, ps), dtype=bool)
        for r in range(B):
            for j in range(n):
                if (r, j) not in skipped:
                    written[table[r, pos[r][j] // ps], pos[r][j] % ps] = True
                assert torch.all(q_out[r, j] == 7.0).item() == ((r, j) in skipped and want[0] != 2)
        w = torch.from_numpy(written).cuda()
        for c in (kc, vc):
            assert torch.all(c.transpose(1, 2)[~w] == 9.0)
            assert not torch.any(torch.all(c.transpose(1, 2)[w] == 9.0, -1))
        assert qsa.check_errors(ws)[0] == qsa.OK


# --------------------------------------------------------------------------
# reading back
# --------------------------------------------------------------------------
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("B,n,hk,D,ps", [(1, 1, 2, 128, 64), (3, 45, 2, 128, 64), (2, 300, 1, 64, 16), (2, 33, 8, 256, 256)])
def test_gather(qsa, kv, B, n, hk, D, ps):
    tokens = [n + 17 * r for r in range(B)]
    table, num_pages = R.page_table(tokens, ps, 4)
    kc, vc, ks, vs = R.make_cache(num_pages, hk, ps, D, kv, 31)
    rng = np.random.RandomState(8)
    pos = np.stack([rng.randint(0, t, n) for t in tokens])  # any order, some twice
    if n > 4:
        pos[0, 3] = pos[-1, n - 1] = -1
    d = _dims(qsa, B, table.shape[1], num_pages, kv, hq=hk, hk=hk, D=D, ps=ps)
    ws = qsa.make_kv_workspace(d)
    ko, vo = (torch.full((B, n, hk, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qsa.kv_gather(d, kc, vc, ks, vs, table.cuda(), _i32(pos), ko, vo, ws)
    _ok(qsa, ws)
    for c, s, o in ((kc, ks, ko), (vc, vs, vo)):
        val = c.cpu() if kv == "bf16" else c.cpu().view(torch.float8_e4m3fn).float() * s.cpu().view(1, -1, 1, 1)
        for r in range(B):
            p = pos[r]
            want = val[table.numpy()[r, p // ps].astype(np.int64), :, p % ps].to(torch.bfloat16)
            want[torch.from_numpy(p < 0)] = 7.0
            assert torch.equal(o[r].cpu(), want)


def test_gather_reports_and_skips(qsa):
    kc, vc, ks, vs = R.make_cache(3, 2, 16, 64, "fp8", 5)
    d = _dims(qsa, 2, 2, 3, "fp8", hq=2, hk=2, D=64, ps=16)
    ws = qsa.make_kv_workspace(d)
    table = _i32([[0, 1], [2, -1]])
    for pos, want, bad in (([[0, 32], [1, 2]], (1, 0, 1, 32), (0, 1)), ([[0, 1], [16, 2]], (2, 1, 0, -1), (1, 0)),
                           ([[0, -5], [1, 2]], (1, 0, 1, -5), (0, 1))):
        ko, vo = (torch.full((2, 2, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        qsa.kv_gather(d, kc, vc, ks, vs, table, _i32(pos), ko, vo, ws)
        assert qsa.check_errors(ws) == (qsa.ERR_BAD_INDEX, want)
        for o in (ko, vo):
            for r in range(2):
                for j in range(2):
                    assert torch.all(o[r, j] == 7.0).item() == ((r, j) == bad)


# --------------------------------------------------------------------------
# dense attention
# --------------------------------------------------------------------------
def _attn_tol(ref, mag, lse, qk, D, kv, small):
    """Output: half a BF16 step of the result; every weight is off by its own
    rounding, by the score's error as an exponent, and by the exponential and
    the sums (2^-18 covers a few thousand FP32 steps taken in trees); the
    score's error is that of an FP32 sum of D products, at most 2^-23 of the
    sum of their magnitudes for each of about D / 8 + 8 partial sums. lse: the
    score's error and a few FP32 steps.

    The weights' rounding: 2^-8 in BF16. With an E4M3 cache a weight p is hi +
    lo / 32, two E4M3 codes: hi is off by at most 2^-4 p, and lo holds that
    rest to 2^-4 of it, so 2^-8 p in all; below the normal codes lo is off by
    up to 2^-10, that is 2^-15 after the division, where the row's largest
    weight is at least 2^6: at most 2^-21 of the largest weight for every
    position."""
    eps_s = (D / 8 + 8) * 2.0 ** -23 * qk
    w = 2.0 ** -8 + 2.0 ** -18
    tiny = 2.0 ** -21 * small if kv == "fp8" else 0.0
    fin = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return 2.0 ** -8 * np.abs(ref) + (w + 2 * eps_s)[..., None] * mag + tiny, eps_s + 2.0 ** -18 * (1 + fin)


def _attn_case(qsa, ctx, n_q, hq, hk, D, ps, kv, window=0, q_pos=None, seed=41, mutate=None, sm_scale=0.0,
               stream=None, max_pages=None):
    """Runs paged_attn on requests of ctx tokens (their n_q newest are the
    queries) and compares every row with the reference; returns the state."""
    B = len(ctx)
    table, num_pages = R.page_table([max(c, 1) for c in ctx], ps, seed)
    if max_pages:
        table = torch.nn.functional.pad(table, (0, max_pages - table.shape[1]), value=-7)
    kc, vc, ks, vs = R.make_cache(num_pages, hk, ps, D, kv, seed + 1)
    q = _normal((B, n_q, hq, D), seed + 2)
    if q_pos is None:
        q_pos = [[max(-1, c - n_q + j) for j in range(n_q)] for c in ctx]
    if mutate:
        mutate(kc, vc, q, table)
    d = _dims(qsa, B, table.shape[1], num_pages, kv, n_q, hq, hk, D, ps, sm_scale=sm_scale)
    ws = qsa.make_kv_workspace(d)
    out = torch.full((B, n_q, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, n_q, hq), 7.0, device="cuda")
    args = (d, q, kc, vc, ks, vs, table.cuda(), _i32(q_pos), out, ws)
    qsa.paged_attn(*args, lse=lse, window=window)
    _ok(qsa, ws)
    _compare_attn(args, lse, window)
    return args, lse


def _compare_attn(args, lse, window=0, bad_pages=None):
    d, q, kc, vc, ks, vs, table, q_pos, out, _ = args
    kv = "bf16" if kc.dtype == torch.bfloat16 else "fp8"
    sc = [R.f64(s)[None, :, None] if kv == "fp8" else 1.0 for s in (ks, vs)]
    caches = [R.f64(kc), R.f64(vc)]
    table, q_pos, q64 = table.cpu().numpy(), q_pos.cpu().numpy(), R.f64(q)
    got, got_lse = R.f64(out), R.f64(lse)
    scale = d.sm_scale if d.sm_scale > 0 else 1.0 / math.sqrt(d.head_dim)
    for r in range(d.batch):
        top = int(q_pos[r].max()) + 1
        k, v = (R.rows(c, table[r], top) * s for c, s in zip(caches, sc)) if top > 0 else (None, None)
        for j in range(d.n_q):
            p = int(q_pos[r, j])
            lo = max(0, p - window + 1) if window else 0
            if p < 0:
                assert np.all(got[r, j] == 0) and np.all(got_lse[r, j] == -np.inf), (r, j)
                continue
            ref, rl, mag, qk, small = R.attention(q64[r, j], k, v, scale, lo, p + 1)
            tol, tol_l = _attn_tol(ref, mag, rl, qk, d.head_dim, kv, small)
            err, err_l = np.abs(got[r, j] - ref), np.abs(got_lse[r, j] - rl)
            assert np.all(err <= tol), (r, j, err.max(), (err - tol).max())
            assert np.all(err_l <= tol_l), (r, j, err_l.max())


HEADS = [(16, 2, 128), (8, 1, 64), (4, 4, 256), (12, 4, 64), (7, 1, 128), (32, 2, 128), (24, 1, 256), (40, 1, 64)]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hk,D", HEADS)
@pytest.mark.parametrize("n_q", [1, 4])
def test_attn_heads(qsa, kv, hq, hk, D, n_q):
    _attn_case(qsa, [333, 70, 1500], n_q, hq, hk, D, 64, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_attn_lengths(qsa, kv, ps, window):
    # one position, sizes round every tile and page border, empty requests
    ctx = [1, 2, 3, 15, 16, 17, 31, 33, 63, 64, 65, 66, 127, 128, 129, 191, 193, 255, 256, 257, 0, 700]
    _attn_case(qsa, ctx, 3, 8, 2, 128, ps, kv, window=window)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("B,ctx,window,n_q", [(1, 20011, 0, 4), (1, 9000, 4097, 1), (5, 6007, 0, 2), (40, 900, 0, 1)])
def test_attn_long_and_wide(qsa, kv, B, ctx, window, n_q):
    _attn_case(qsa, [ctx - 131 * r % 500 for r in range(B)], n_q, 16, 2, 128, 64, kv, window=window)


@pytest.mark.parametrize("D,B", [(128, 300), (64, 700), (128, 256), (256, 257)])
def test_attn_many_requests(qsa, D, B):
    # more requests than threads, empty ones among them; one long request among
    # short ones, cut into many pieces
    ctx = [(37 * r) % 190 if r % 7 else 0 for r in range(B)]
    ctx[B // 2] = 9000
    _attn_case(qsa, ctx, 1, 4, 2, D, 16, "bf16")


@pytest.mark.parametrize("gap", [1, 31, 32, 33, 64, 1000, 262144])
def test_attn_empty_requests_between(qsa, gap):
    # runs of free slots between live requests, one of them longer than any: the
    # CTA that has live ones on both sides gets past them (a second's wait of its
    # roles for one another is not near; one slot after the other, the longest took
    # 86 ms)
    import time

    ps, D, hq = 16, 64, 2
    live = np.unique(np.r_[np.arange(400), 400 + gap + np.arange(3), 403 + 2 * gap + 33 * np.arange(4)])
    B = int(live[-1]) + 1 + gap % 50
    kc, vc, ks, vs = R.make_cache(8, 1, ps, D, "bf16", 5)
    d = _dims(qsa, B, 4, 8, "bf16", 1, hq, 1, D, ps)
    ws, q = qsa.make_kv_workspace(d), _normal((1, 1, hq, D), 6).expand(B, 1, hq, D).contiguous()
    table = _i32([[3, 0, 7, 5]]).repeat(B, 1)
    pos = torch.full((B, 1), -1, dtype=torch.int32)
    pos[live, 0] = torch.from_numpy((live % 7 * 8 + 2).astype(np.int32))
    pos = pos.cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((B, 1, hq), 7.0, device="cuda")
    took = []
    for _ in range(3):
        torch.cuda.synchronize()
        t = time.time()
        qsa.paged_attn(d, q, kc, vc, None, None, table, pos, out, ws, lse=lse)
        torch.cuda.synchronize()
        took.append(time.time() - t)
    _ok(qsa, ws)
    assert min(took) < 0.04, took
    seen = torch.from_numpy(live).cuda()
    _compare_attn((_dims(qsa, len(live), 4, 8, "bf16", 1, hq, 1, D, ps), q[seen], kc, vc, ks, vs, table[seen], pos[seen],
                   out[seen], ws), lse[seen])
    rest = torch.ones(B, dtype=torch.bool, device="cuda")
    rest[seen] = False
    assert torch.all(out[rest] == 0) and torch.all(lse[rest] == -math.inf)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attn_positions_of_any_order(qsa, kv):
    # queries far apart, the same position twice, padding rows between, a page
    # table wider than the requests with ids in it that nothing may read
    pos = [[5, 900, -1, 0], [-1, -1, -1, -1], [1000, 10, 1000, 500]]
    for window in (0, 300):
        _attn_case(qsa, [901, 64, 1001], 4, 16, 2, 128, 32, kv, window=window, q_pos=pos, max_pages=200)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hk,n_q", [(1024, 1, 4), (1023, 1, 1), (512, 512, 2), (1024, 256, 4)])
def test_attn_most_heads(qsa, kv, hq, hk, n_q):
    # many blocks of rows of one KV head, and more units than positions
    _attn_case(qsa, [130, 3], n_q, hq, hk, 64, 32, kv)


@pytest.mark.parametrize("window", [129, 2 ** 31 - 1])
def test_attn_window_past_the_context(qsa, window):
    args, lse = _attn_case(qsa, [128, 5], 2, 16, 2, 128, 64, "bf16", window=window)
    whole, lse2 = _attn_case(qsa, [128, 5], 2, 16, 2, 128, 64, "bf16")
    assert torch.equal(args[8], whole[8]) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("sm_scale", [1e-3, 3.0])
def test_attn_scale(qsa, kv, sm_scale):
    _attn_case(qsa, [500, 130], 2, 16, 2, 128, 64, kv, sm_scale=sm_scale)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("factor", [1e5, 1e-6])
def test_attn_query_magnitudes(qsa, kv, factor):
    # queries outside FP16's range keep their BF16 values with either cache
    def scale_q(kc, vc, q, table):
        q.mul_(factor)

    _attn_case(qsa, [300, 90], 4, 16, 2, 128, 64, kv, mutate=scale_q, sm_scale=0.05 / factor)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_what_is_masked_never_arrives(qsa, kv, bad, D):
    # everything that a query does not see is NaN or infinite: slots behind the
    # last position, positions before the window, the spare page; and position
    # p_j + 1 .. p_3 for the earlier queries of a verify step
    if kv == "fp8" and not math.isnan(bad):
        pytest.skip("E4M3 has no infinities")
    ctx, n_q, window, ps = [77, 130, 66], 4, 40, 16
    code = torch.tensor(bad).to(torch.bfloat16) if kv == "bf16" else 0x7F
    keep = {}

    def poison(kc, vc, q, table):
        seen = torch.zeros(kc.shape[0], ps, dtype=torch.bool)
        for r, c in enumerate(ctx):
            lo = max(0, c - n_q - window + 1)
            p = np.arange(lo, c)
            seen[torch.from_numpy(table.numpy()[r, p // ps].astype(np.int64)), torch.from_numpy(p % ps)] = True
        for c in (kc, vc):
            c.transpose(1, 2)[~seen.cuda()] = code
        keep["cache"] = (kc, vc)

    args, lse = _attn_case(qsa, ctx, n_q, 16, 2, D, ps, kv, window=window, mutate=poison)
    # now the newest token and the oldest of the window: rows that see neither keep their bits
    clean, clean_lse = args[8].clone(), lse.clone()
    table = args[6].cpu().numpy()
    for r, c in enumerate(ctx):
        for p in (c - 1, c - n_q - window + 1):
            if p >= 0:
                for x in keep["cache"]:
                    x[int(table[r, p // ps]), :, p % ps] = code
    qsa.paged_attn(*args, lse=lse, window=window)
    _ok(qsa, args[9])
    out, lse = args[8].float(), lse
    for r, c in enumerate(ctx):
        for j in (1, 2):
            if c - n_q - window + 1 >= 0 or j == 1 or True:
                assert torch.isfinite(out[r, j]).all() and torch.isfinite(lse[r, j]).all(), (r, j)
                err = (out[r, j] - clean[r, j].float()).abs().max().item()
                assert err <= 2.0 ** -7 * clean[r, j].float().abs().max().item(), (r, j, err)
                assert (lse[r, j] - clean_lse[r, j]).abs().max().item() <= 2.0 ** -16 * 10
        assert torch.isnan(out[r, 3]).all()  # it sees the newest token (0 * inf and inf - inf are NaN)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attn_not_finite_queries_stay_in_their_rows(qsa, kv, bad):
    # a query with an infinity or NaN gives NaN (inf - inf, 0 * inf), the others
    # the same bits as without it
    args, lse = _attn_case(qsa, [300, 40], 4, 16, 2, 128, 64, kv)
    clean, clean_lse = args[8].clone(), lse.clone()
    args[1][0, 2, 5, 77] = bad
    args[1][1, 0, 15, 0] = bad
    qsa.paged_attn(*args, lse=lse)
    _ok(qsa, args[9])
    hit = torch.zeros((2, 4, 16), dtype=torch.bool, device="cuda")
    hit[0, 2, 5] = hit[1, 0, 15] = True
    assert torch.isnan(args[8][hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(args[8][~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


def test_attn_infinite_values_arrive(qsa):
    # an infinite V that a row does see gives the infinity that arithmetic gives
    def plant(kc, vc, q, table):
        vc[int(table[0, 1]), 0, 3, 5] = math.inf

    B, hq = 1, 8
    table, num_pages = R.page_table([200], 64, 1)
    kc, vc, ks, vs = R.make_cache(num_pages, 1, 64, 128, "bf16", 2)
    q = _normal((1, 4, hq, 128), 3)
    plant(kc, vc, q, table)
    d = _dims(qsa, B, table.shape[1], num_pages, "bf16", 4, hq, 1)
    ws = qsa.make_kv_workspace(d)
    out = torch.empty_like(q)
    # query 0 and 1 do not see position 67, 2 and 3 do
    qsa.paged_attn(d, q, kc, vc, None, None, table.cuda(), _i32([[66, 60, 67, 199]]), out, ws)
    _ok(qsa, ws)
    assert torch.isfinite(out[0, :2]).all()
    assert torch.all(out[0, 2:, :, 5] == math.inf)
    rest = torch.ones(128, dtype=torch.bool)
    rest[5] = False
    assert torch.isfinite(out[0, 2:, :, rest]).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attn_lowest_scores(qsa, kv):
    # scores near the lowest FP32 value are still scores: 1.44 x 2.6 x 2^126 in
    # the exp2 domain is -3.19e38
    args, lse = _attn_case(qsa, [1, 2, 700], 1, 16, 2, 64, 64, kv, sm_scale=2.6)
    d, q, kc, vc, ks, vs = args[:6]
    q.zero_()
    kc.zero_()
    # q . k = -2^126 everywhere: BF16 -2^63 x 2^63, E4M3 -2^119 x 2^7 (code 0x70)
    q[..., 0] = -2.0 ** (63 if kv == "bf16" else 119)
    kc[..., 0] = 2.0 ** 63 if kv == "bf16" else 0x70
    if kv == "fp8":
        ks.fill_(1.0)
    qsa.paged_attn(*args, lse=lse)
    got, pos = R.f64(args[8]), args[7].cpu().numpy()
    v = R.f64(vc) * (R.f64(vs)[None, :, None, None] if kv == "fp8" else 1.0)
    table = args[6].cpu().numpy()
    for r in range(3):
        t = np.arange(pos[r, 0] + 1)
        rows = v[table[r][t // 64], :, t % 64]  # [t][H_kv][D]
        want, size = rows.mean(axis=0), np.abs(rows).mean(axis=0)
        # equal weights, all exact: FP32 sums (2^-18 covers 700 of them) and one rounding
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size
        assert np.all(np.abs(got[r, 0] - np.repeat(want, 8, axis=0)) <= np.repeat(tol, 8, axis=0)), r
    assert np.allclose(R.f64(lse), -2.6 * 2.0 ** 126, rtol=1e-6)
    _ok(qsa, args[9])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("up", [24, 28, 32, 60])
def test_attn_huge_scores(qsa, kv, up):
    # scores of 2^up and more, whose FP32 steps are of any size: one weight is
    # all there is (the reference's gap of a row's two largest scores says for
    # which rows), and a row of one position gives its value
    args, lse = _attn_case(qsa, [1, 2, 130, 700], 2, 16, 2, 128, 64, kv)
    d, q, kc, vc, ks, vs = args[:6]
    q.mul_(2.0 ** up)
    qsa.paged_attn(*args, lse=lse)
    k, v = R.f64(kc), R.f64(vc)
    if kv == "fp8":
        k, v = k * R.f64(ks)[None, :, None, None], v * R.f64(vs)[None, :, None, None]
    got, got_lse, q64, pos, table = R.f64(args[8]), R.f64(lse), R.f64(q), args[7].cpu().numpy(), args[6].cpu().numpy()
    sure = 0
    for r, j in np.ndindex(pos.shape):
        t = np.arange(pos[r, j] + 1)
        if not len(t):
            continue
        for h in range(16):
            rows = k[table[r][t // 64], h // 8, t % 64]
            s = rows @ q64[r, j, h] / math.sqrt(128)
            best, size = s.argmax(), (np.abs(rows) @ np.abs(q64[r, j, h])).max() / math.sqrt(128)
            # FP32 sums of 128 products, Q down to 2^-23 of its largest value: 2^-15 of the sum of magnitudes
            assert abs(got_lse[r, j, h] - s[best]) <= 2.0 ** -15 * size + 10
            if np.delete(s, best).max(initial=-np.inf) < s[best] - 2.0 ** -14 * size - 40:
                want = v[table[r][t[best] // 64], h // 8, t[best] % 64]
                # one weight: the roundings of P and of the output, 2^-8 each
                assert np.all(np.abs(got[r, j, h] - want) <= (2.0 ** -7 + 2.0 ** -14) * np.abs(want) + 2.0 ** -18), (r, j, h)
                sure += 1
    assert sure > 90  # of 7 x 16
    _ok(qsa, args[9])


def test_attn_reports_and_skips(qsa):
    ps, hk, D = 16, 2, 128
    table, num_pages = R.page_table([100, 100], ps, 9)
    kc, vc, ks, vs = R.make_cache(num_pages, hk, ps, D, "bf16", 10)
    q = _normal((2, 2, 16, D), 11)
    d = _dims(qsa, 2, table.shape[1], num_pages, "bf16", 2, 16, hk, D, ps)
    ws = qsa.make_kv_workspace(d)
    out, lse = torch.empty_like(q), torch.empty((2, 2, 16), device="cuda")
    cap = table.shape[1] * ps
    for p, in ((cap,), (-2,)):
        qsa.paged_attn(d, q, kc, vc, ks, vs, table.cuda(), _i32([[98, 99], [p, 50]]), out, ws, lse=lse)
        assert qsa.check_errors(ws) == (qsa.ERR_BAD_INDEX, (1, 1, 0, p))
        good = torch.tensor([[98, 99], [-1, 50]])
        _compare_attn((d, q, kc, vc, ks, vs, table.cuda(), good, out, ws), lse)
    for bad in (num_pages, -1, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 2] = bad
        qsa.paged_attn(d, q, kc, vc, ks, vs, t.cuda(), _i32([[98, 99], [98, 99]]), out, ws, lse=lse)
        st, info = qsa.check_errors(ws)
        assert st == qsa.ERR_BAD_INDEX and info[0] == 2 and info[1] == 1 and info[3] == bad
        # the same as a cache where those 16 positions weigh nothing
        keep = np.r_[0:32, 48:100]
        k, v = (R.rows(R.f64(c), table.numpy()[1], 100)[keep] for c in (kc, vc))
        for j in range(2):
            n = len(keep) - 1 + j
            ref, rl, mag, qk, small = R.attention(R.f64(q[1, j]), k, v, 1 / math.sqrt(D), 0, n)
            tol, tol_l = _attn_tol(ref, mag, rl, qk, D, "bf16", small)
            assert np.all(np.abs(R.f64(out[1, j]) - ref) <= tol)
            assert np.all(np.abs(R.f64(lse[1, j]) - rl) <= tol_l)
    # a request whose pages are all bad has nothing to attend to
    t = table.clone()
    t[1] = -1
    qsa.paged_attn(d, q, kc, vc, ks, vs, t.cuda(), _i32([[98, 99], [98, 99]]), out, ws, lse=lse)
    assert qsa.check_errors(ws)[0] == qsa.ERR_BAD_INDEX
    assert torch.all(out[1] == 0) and torch.all(lse[1] == -math.inf)


@pytest.mark.parametrize("ps", [16, 64, 256])
def test_attn_pages_outside_the_window_are_not_looked_up(qsa, ps):
    # pages that slid out of the window were given back, those behind the last
    # position do not exist yet: their ids mean nothing and nothing is reported
    ctx, window, n_q = [1000, 333], 100, 2

    def free(kc, vc, q, table):
        for r, c in enumerate(ctx):
            lo = c - n_q - window + 1
            table[r, :lo // ps] = -5
            table[r, -(-c // ps):] = 1 << 30

    _attn_case(qsa, ctx, n_q, 16, 2, 128, ps, "bf16", window=window, mutate=free)


def test_attn_closed_forms(qsa):
    # one position: its V row bit for bit; keys of zero: the mean of V
    D = 128
    table, num_pages = R.page_table([1, 700], 64, 12)
    kc, vc, ks, vs = R.make_cache(num_pages, 2, 64, D, "bf16", 13)
    kc.zero_()
    q = _normal((2, 1, 16, D), 14)
    d = _dims(qsa, 2, table.shape[1], num_pages)
    ws = qsa.make_kv_workspace(d)
    out, lse = torch.empty_like(q), torch.empty((2, 1, 16), device="cuda")
    qsa.paged_attn(d, q, kc, vc, ks, vs, table.cuda(), _i32([[0], [699]]), out, ws, lse=lse)
    _ok(qsa, ws)
    row = vc[int(table[0, 0]), :, 0]
    assert torch.equal(out[0, 0], row.repeat_interleave(8, 0)) and torch.all(lse[0] == 0)
    mean = R.rows(R.f64(vc), table.numpy()[1], 700).mean(0).repeat(8, 0)
    assert np.all(np.abs(R.f64(out[1, 0]) - mean) <= 2.0 ** -8 * np.abs(mean) + 2.0 ** -17)
    assert (lse[1] - math.log(700)).abs().max().item() <= 2.0 ** -20 * 8


@pytest.mark.parametrize("v_kind", ["ones", "apart", "alternating", "normal"])
@pytest.mark.parametrize("kv,D,n_q,T,gap", [
    ("bf16", 128, 1, 61204, 14.6), ("fp8", 128, 1, 61204, 14.6), ("fp8", 128, 1, 61204, 14.2),
    ("fp8", 128, 4, 61204, 14.0), ("fp8", 64, 1, 400001, 14.6), ("fp8", 64, 4, 61203, 13.0),
    ("fp8", 256, 2, 61204, 15.5), ("fp8", 64, 2, 1000000, 14.6), ("fp8", 64, 1, 1000000, 17.3)])
def test_attn_long_flat_tail(qsa, kv, D, n_q, T, gap, v_kind):
    # one key `gap` nats above a long tail of equal ones: each weight of the tail
    # is next to nothing, their sum is not. As many requests as give every CTA
    # about a whole unit (they read the same pages), since a piece without the
    # large key has a reference of its own.
    #
    # Tolerance: half a BF16 step of the result (2^-8), the weights' own rounding
    # (2^-8 of each), and with an E4M3 cache what weights below 2^-6 (the largest
    # is at least 2^6) lose: each is off by less than a step of 2^-14, up or down
    # with mean zero, a variance of at most 2^-14 times the weight. Over a tail
    # of sum S that is sqrt(2^-14 S) of S + 2^6 or more, at most 2^-11; six times
    # that are allowed. Nothing in it grows with the number of positions.
    ps, hk = 256, 2
    B = -(-torch.cuda.get_device_properties(0).multi_processor_count // hk)
    pages = -(-T // ps)
    code = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    g = torch.Generator("cuda").manual_seed(17)

    def cache(x):  # [T] or [T][D] values that the type holds, the same for every head
        c = torch.zeros((pages * ps, D), device="cuda")
        c[:T] = x if x.dim() == 2 else x[:, None]
        c = c.to(code).view(pages, 1, ps, D).expand(pages, hk, ps, D).contiguous()
        return c if kv == "bf16" else c.view(torch.uint8)

    k = torch.zeros((T, D), device="cuda")
    k[0, 0] = 1.0
    v = torch.ones((T, D), device="cuda")
    if v_kind == "apart":
        v[0] = -1.0
    elif v_kind == "alternating":
        v[::2] = -0.5
    elif v_kind == "normal":
        v = torch.randn((T, D), generator=g, device="cuda") + 0.5
    kc, vc = cache(k), cache(v)
    v64 = R.f64(vc.transpose(1, 2)[:, :, 0].reshape(pages * ps, D)[:T])
    d = _dims(qsa, B, pages, pages, kv, n_q, 16, hk, D, ps, sm_scale=gap)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0)
    kc, vc = kc.flip(0).contiguous(), vc.flip(0).contiguous()
    q = torch.zeros((B, n_q, 16, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    pos = _i32([[T - n_q + j for j in range(n_q)]] * B)
    one, ws = torch.ones(hk, device="cuda"), qsa.make_kv_workspace(d)
    out, lse = torch.empty_like(q), torch.empty((B, n_q, 16), device="cuda")
    qsa.paged_attn(d, q, kc, vc, one, one, table.repeat(B, 1), pos, out, ws, lse=lse)
    _ok(qsa, ws)
    for j in range(n_q):
        n = T - n_q + j + 1
        w = np.full(n, math.exp(-float(np.float32(gap))))
        w[0] = 1.0
        want, big = w @ v64[:n] / w.sum(), np.abs(v64[:n]).max(0)
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 6 * 2.0 ** -11 + 2.0 ** -18) * big
        err = np.abs(R.f64(out[:, j]) - want)
        assert np.all(err <= tol), (j, err.max(), (err - tol).max())
        # a thread adds its position of up to 256 tiles to its part of the sum in turn: FP32 additions, each off
        # by at most 2^-24 of the part (the largest key's: 2^6, to which a tail weight of less than 2^-18 adds nothing)
        sums = 256 * 2.0 ** -24
        assert np.abs(R.f64(lse[:, j]) - gap - math.log(w.sum())).max() <= 2.0 ** -18 * (1 + gap) + sums


@pytest.mark.parametrize("kv,D,n_q,hq,T,window", [
    ("bf16", 128, 1, 16, 61204, 0), ("bf16", 64, 1, 16, 400001, 0), ("bf16", 64, 4, 32, 1000000, 0),
    ("bf16", 256, 1, 16, 400001, 350000), ("fp8", 128, 4, 16, 1000000, 0), ("fp8", 64, 4, 32, 1000000, 700001),
    ("fp8", 64, 1, 16, 4000000, 0), ("fp8", 256, 4, 32, 400001, 0)])
def test_attn_long_sums(qsa, kv, D, n_q, hq, T, window):
    # Keys of every size and the same value at every position: whatever the
    # weights, the output is that value, bit for bit, as long as sums over a unit
    # that one CTA has to itself are right to 2^-10 or so (half a BF16 step of 1.75
    # is 2^-8.8 of it; the weights' own roundings, at most 2^-8 each, are as often
    # up as down, and T of them leave next to nothing).
    ps, hk = 256, 2
    B = -(-torch.cuda.get_device_properties(0).multi_processor_count // (hk * (2 if hq * n_q > 128 else 1)))
    pages = -(-T // ps)
    code = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    k = torch.randn((pages, 1, ps, D), generator=torch.Generator("cuda").manual_seed(18), device="cuda").to(code)
    v = torch.full((pages, hk, ps, D), 1.75, device="cuda").to(code)
    one = torch.ones(hk, device="cuda")
    q = torch.randn((1, 1, hq, D), generator=torch.Generator("cuda").manual_seed(19), device="cuda").to(torch.bfloat16)
    s = k[:, 0].reshape(-1, D)[:T].double() @ q[0, 0].double().t() * float(np.float32(1 / math.sqrt(D)))
    kc, vc = k.expand(pages, hk, ps, D).contiguous(), v
    if kv == "fp8":
        kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
    d = _dims(qsa, B, pages, pages, kv, n_q, hq, hk, D, ps)
    pos, ws = _i32([[T - n_q + j for j in range(n_q)]] * B), qsa.make_kv_workspace(d)
    q = q.expand(B, n_q, hq, D).contiguous()
    out, lse = torch.empty_like(q), torch.empty((B, n_q, hq), device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1)
    qsa.paged_attn(d, q, kc, vc, one, one, table, pos, out, ws, lse=lse, window=window)
    _ok(qsa, ws)
    assert torch.all(out == 1.75), (out.min().item(), out.max().item())
    for j in range(n_q):
        n = T - n_q + j + 1
        want = torch.logsumexp(s[max(0, n - window) if window else 0:n], 0)
        # the scores' FP32 sums (see _attn_tol) and those of the weights
        size = (k[:, 0].reshape(-1, D)[:n].float().abs() @ q[0, 0].float().abs().t()).max().item() / math.sqrt(D)
        assert (lse[:, j].double() - want).abs().max().item() <= (D / 8 + 8) * 2.0 ** -23 * size + 2.0 ** -16


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("fp8", 128), ("bf16", 256), ("fp8", 64)])
@pytest.mark.parametrize("T,window", [(32768, 0), (32770, 0), (65537, 0), (70000, 33000)])
def test_attn_long_units_end_to_end(qsa, kv, D, T, window):
    # units long enough for more than one run of tiles in a CTA, the last run of
    # one tile or of an edge alone, with the newest token's V NaN: only the last
    # query sees it. Every request is the same, so is every answer.
    ps, hk, hq, n_q = 64, 2, 16, 4
    B = -(-torch.cuda.get_device_properties(0).multi_processor_count // hk)
    table, pages = R.page_table([T], ps, 23)
    kc, vc, ks, vs = R.make_cache(pages, hk, ps, D, kv, 24)
    d = _dims(qsa, B, table.shape[1], pages, kv, n_q, hq, hk, D, ps)
    q = _normal((1, n_q, hq, D), 25).expand(B, n_q, hq, D).contiguous()
    pos, ws = _i32([[T - n_q + j for j in range(n_q)]] * B), qsa.make_kv_workspace(d)
    out, lse = torch.empty_like(q), torch.empty((B, n_q, hq), device="cuda")
    args = [q, kc, vc, ks, vs, table.cuda().repeat(B, 1), pos, out, ws]
    qsa.paged_attn(d, *args, lse=lse, window=window)
    _ok(qsa, ws)
    clean = out.clone()
    # (the units' first and last pieces are cut at other places: equal up to the roundings)
    one = _dims(qsa, 1, table.shape[1], pages, kv, n_q, hq, hk, D, ps)
    for r in (0, B // 2 + 1):
        _compare_attn((one, q[:1], kc, vc, ks, vs, table.cuda(), pos[:1], out[r:r + 1], ws), lse[r:r + 1], window)
    vc[int(table[0, (T - 1) // ps]), :, (T - 1) % ps] = math.nan if kv == "bf16" else 0x7F
    qsa.paged_attn(d, *args, lse=lse, window=window)
    _ok(qsa, ws)
    assert torch.isnan(out[:, 3]).all()
    err = (out[:, :3].float() - clean[:, :3].float()).abs().max().item()
    assert err <= 2.0 ** -7 * clean.float().abs().max().item(), err


def test_attn_without_lse_and_repeated(qsa):
    # the same bits on every call, with and without lse, whatever ws held before
    args, lse = _attn_case(qsa, [3000, 41, 1, 777], 4, 16, 2, 128, 64, "fp8")
    first, first_lse = args[8].clone(), lse.clone()
    for k in range(4):
        args[8].fill_(3.0)
        lse.fill_(3.0)
        if k:
            args[9][256:].random_(0, 256)
        qsa.paged_attn(*args, lse=lse if k % 2 else None)
        assert torch.equal(args[8], first)
        assert not k % 2 or torch.equal(lse, first_lse)
    _ok(qsa, args[9])


# --------------------------------------------------------------------------
# streams, graphs, far offsets, and the operators together
# --------------------------------------------------------------------------
def test_other_stream_and_graph(qsa):
    # a step (append, attention) on a side stream, captured and replayed with
    # new inputs in the same buffers, against direct calls
    B, n_q, ps = 3, 4, 64
    ctx = [500, 64, 1301]
    table, num_pages = R.page_table(ctx, ps, 51)
    d = _dims(qsa, B, table.shape[1], num_pages, "fp8", n_q)
    kc, vc, ks, vs = R.make_cache(num_pages, 2, ps, 128, "fp8", 52)
    pt, pos = table.cuda(), _i32([[c - n_q + j for j in range(n_q)] for c in ctx])
    rope = qsa.make_rope(128)
    qkv = _normal((B, n_q, 20, 128), 53)
    ws = qsa.make_kv_workspace(d)
    q_rot, out = (torch.empty((B, n_q, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(stream=None):
        qsa.kv_append(d, qkv[:, :, 16:18], qkv[:, :, 18:], kc, vc, ks, vs, pt, pos, ws, rope=rope, q=qkv[:, :, :16],
                      q_out=q_rot, stream=stream)
        qsa.paged_attn(d, q_rot, kc, vc, ks, vs, pt, pos, out, ws, stream=stream)

    side = torch.cuda.Stream()
    inputs = [qkv.clone(), _normal(qkv.shape, 54), _normal(qkv.shape, 55)]
    want = []
    for x in inputs:
        qkv.copy_(x)
        step()
        want.append((out.clone(), q_rot.clone(), kc.clone(), vc.clone()))
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for x, ref in zip(inputs, want):
        qkv.copy_(x)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, q_rot, kc, vc), ref):
            assert torch.equal(a, b)
        out.zero_()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            step()
        step(stream=side)  # named, from another current stream
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0])
    _ok(qsa, ws)


def test_what_follows_waits_for_whole_units(qsa):
    # every CTA has one whole unit, so the joining kernel has nothing to join:
    # it still must not end before the kernel that writes the rows
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B, n = sms // 2, 8192
    per = n // 256
    d = _dims(qsa, B, per, B * per, "bf16", 1, ps=256)
    kc, vc = (torch.randn((B * per, 2, 256, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    pt = torch.randperm(B * per, device="cuda").to(torch.int32).view(B, per)
    pos = torch.full((B, 1), n - 1, dtype=torch.int32, device="cuda")
    q, ws = _normal((B, 1, 16, 128), 57), qsa.make_kv_workspace(d)
    out, turned = torch.empty_like(q), torch.empty_like(q)
    rope = qsa.make_rope(128)

    def step():
        qsa.paged_attn(d, q, kc, vc, None, None, pt, pos, out, ws)
        qsa.rope(rope, out, pos, turned)

    step()
    torch.cuda.synchronize()
    want = out.clone(), turned.clone()
    assert not torch.isnan(out).any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        kept = out.clone()
    for _ in range(5):
        out.fill_(math.nan)
        step()
        got = out.clone()
        assert torch.equal(got, want[0]) and torch.equal(turned, want[1])
        out.fill_(math.nan)
        qsa.paged_attn(d, q, kc, vc, None, None, pt, pos, out, ws)
        assert torch.equal(out.clone(), want[0])
        out.fill_(math.nan)
        graph.replay()
        assert torch.equal(kept, want[0]) and torch.equal(turned, want[1])
    _ok(qsa, ws)


def test_captured_branches(qsa):
    # two branches of a captured graph (one rotates and appends, one reads
    # older rows back) that meet in the attention
    B, ps = 2, 64
    ctx = [500, 130]
    table, num_pages = R.page_table(ctx, ps, 61)
    d = _dims(qsa, B, table.shape[1], num_pages)
    kc, vc, _, _ = R.make_cache(num_pages, 2, ps, 128, "bf16", 62)
    pt, pos = table.cuda(), _i32([[c - 1] for c in ctx])
    old = _i32([[3, 77, 400], [0, 128, 5]])
    qkv, rope = _normal((B, 1, 20, 128), 63), qsa.make_rope(128)
    ws, ws2 = qsa.make_kv_workspace(d), qsa.make_kv_workspace(d)
    q_rot, out = (torch.empty((B, 1, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ko, vo = (torch.zeros((B, 3, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(main, other):
        other.wait_stream(main)
        qsa.kv_gather(d, kc, vc, None, None, pt, old, ko, vo, ws2, stream=other)
        qsa.kv_append(d, qkv[:, :, 16:18], qkv[:, :, 18:], kc, vc, None, None, pt, pos, ws, rope=rope,
                      q=qkv[:, :, :16], q_out=q_rot, stream=main)
        main.wait_stream(other)
        qsa.paged_attn(d, q_rot, kc, vc, None, None, pt, pos, out, ws, stream=main)

    side = torch.cuda.Stream()
    step(torch.cuda.current_stream(), side)
    want = [t.clone() for t in (out, ko, vo, kc, vc)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream(), side)
    for _ in range(3):
        for t in (out, ko, vo):
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip((out, ko, vo, kc, vc), want))
    _ok(qsa, ws)
    _ok(qsa, ws2)


def test_two_graphs_share_a_workspace(qsa):
    # replayed in turn, on one stream; and one call's pieces do not need what
    # another call of other dims left there
    args, lse = _attn_case(qsa, [5000, 70, 900], 4, 16, 2, 128, 64, "bf16")
    d2 = qsa.make_dims(3, 1, 1, args[0].max_pages, args[0].num_pages)
    q2 = _normal((3, 1, 16, 128), 99)
    out2, pos2 = torch.empty_like(q2), _i32([[4999], [3], [-1]])
    args2 = (d2, q2, *args[2:7], pos2, out2, args[9])
    qsa.paged_attn(*args2)
    want = args[8].clone(), out2.clone()
    graphs = []
    for a in (args, args2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qsa.paged_attn(*a)
        graphs.append(g)
    for k in (0, 1, 1, 0, 0, 1):
        (args, args2)[k][8].zero_()
        graphs[k].replay()
        assert torch.equal((args, args2)[k][8], want[k])
    _ok(qsa, args[9])


def test_refusals_on_the_device(qsa):
    # through the binding, on real tensors: what is wrong is said, nothing runs
    args, lse = _attn_case(qsa, [100, 7], 2, 16, 2, 128, 64, "fp8")
    d, q, kc, vc, ks, vs, pt, pos, out, ws = args
    before = out.clone()

    def attn(err, match, **kw):
        a = dict(q=q, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, page_table=pt, q_pos=pos, out=out, ws=ws, lse=lse)
        a.update(kw)
        with pytest.raises(err, match=match):
            qsa.paged_attn(d, **a)

    attn(TypeError, "q: dtype", q=q.half())
    attn(TypeError, "k_cache: dtype", k_cache=kc.view(torch.int8))
    attn(ValueError, "q: shape", q=q[:1])
    attn(ValueError, "out must be contiguous", out=torch.empty_like(q).transpose(0, 1).contiguous().transpose(0, 1))
    attn(ValueError, "lse: shape", lse=lse[:, :, :8])
    attn(TypeError, "q_pos: dtype", q_pos=pos.long())
    attn(ValueError, "CUDA", page_table=pt.cpu())
    attn(TypeError, "k_scale must be a tensor", k_scale=None)
    attn(ValueError, "window", window=-1)
    attn(ValueError, "window", window=1 << 31)
    attn(ValueError, "ws must be", ws=ws.cpu())
    attn(qsa.QSAError, "WORKSPACE", ws=ws[:256])
    attn(qsa.QSAError, "WORKSPACE", ws=ws[8:])
    rope = qsa.make_rope(128)
    k = _normal((2, 2, 2, 128), 1)
    for err, match, kw in [
        (ValueError, "last dimension", dict(k=_normal((2, 2, 128, 2), 1).transpose(2, 3))),
        (ValueError, "k: shape", dict(k=k[:, :, :1])),
        (TypeError, "v: dtype", dict(v=k.float())),
        (ValueError, "q needs", dict(q=q)),
        (ValueError, "q needs", dict(q=q, q_out=q, rope=None)),
        (TypeError, "make_rope", dict(rope=1)),
        (ValueError, "pos: shape", dict(pos=pos[:, :1].contiguous())),
        (qsa.QSAError, "INVALID_ARG", dict(q=q, q_out=q.as_strided(q.shape, (0, 2048, 128, 1)))),
        (qsa.QSAError, "INVALID_ARG", dict(rope=qsa.make_rope(256))),
    ]:
        a = dict(k=k, v=k, pos=pos, rope=rope)
        a.update(kw)
        with pytest.raises(err, match=match):
            qsa.kv_append(d, a.pop("k"), a.pop("v"), kc, vc, ks, vs, pt, a.pop("pos"), ws, **a)
    with pytest.raises(qsa.QSAError, match="INVALID_ARG"):  # no token
        qsa.rope(rope, q[:, :0], pos[:, :0], q[:, :0])
    with pytest.raises(ValueError, match="x must be"):
        qsa.rope(rope, q[0], pos, q[0])
    with pytest.raises(ValueError, match="k_out: shape"):
        qsa.kv_gather(d, kc, vc, ks, vs, pt, pos, k[:, :, :1], k, ws)
    _ok(qsa, ws)
    assert torch.equal(out, before)
    # a subclass, a tensor that wants gradients and an empty stream argument are fine
    qsa.paged_attn(d, torch.nn.Parameter(q), kc, vc, ks, vs, pt, pos, out, ws, stream=torch.cuda.current_stream())
    _ok(qsa, ws)
    assert torch.equal(out, before)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_offsets_past_32_bits(qsa, kv):
    # a cache of more than 2^31 elements (2^32 bytes), used at its far end
    ps, hk, D = 64, 2, 128
    num_pages = (1 << 31) // (ps * hk * D) + 40
    dt = torch.bfloat16 if kv == "bf16" else torch.uint8
    kc, vc = (torch.empty((num_pages, hk, ps, D), dtype=dt, device="cuda") for _ in range(2))
    kc[-40:], vc[-40:], ks, vs = R.make_cache(40, hk, ps, D, kv, 61)
    table = torch.arange(num_pages - 10, num_pages, dtype=torch.int32).flip(0).view(1, -1)
    d = _dims(qsa, 1, 10, num_pages, kv, 4)
    ws = qsa.make_kv_workspace(d)
    k, v, q = _normal((1, 4, hk, D), 62), _normal((1, 4, hk, D), 63), _normal((1, 4, 16, D), 64)
    pos = _i32([[600, 601, 602, 603]])
    qsa.kv_append(d, k, v, kc, vc, ks, vs, table.cuda(), pos, ws)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    qsa.kv_gather(d, kc, vc, ks, vs, table.cuda(), pos, ko, vo, ws)
    out, lse = torch.empty_like(q), torch.empty((1, 4, 16), device="cuda")
    qsa.paged_attn(d, q, kc, vc, ks, vs, table.cuda(), pos, out, ws, lse=lse)
    _ok(qsa, ws)
    if kv == "bf16":
        assert torch.equal(ko, k) and torch.equal(vo, v)
    small = (d, q, kc[-40:], vc[-40:], ks, vs, table.cuda() - (num_pages - 40), pos, out, ws)
    _compare_attn(small, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_request_from_prefill_to_decode(qsa, kv):
    # prefill (append a chunk, compress its keys), a sparse verify step and a
    # dense one over the same pages: while every block fits the selection, the
    # sparse step is dense attention. One workspace serves both headers.
    ps, n_ctx, n_q = 64, 1500, 4
    total = n_ctx + n_q
    table, num_pages = R.page_table([total], ps, 71)
    pt = table.cuda()
    d = qsa.make_dims(1, n_q, total // 4, table.shape[1], num_pages, 1, kv)
    kc, vc, ks, vs = R.make_cache(num_pages, 2, ps, 128, kv, 72)
    kc.zero_(), vc.zero_()
    n = max(qsa.workspace_size(d), qsa.kv_workspace_size(d))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    rope = qsa.make_rope(128)
    x = _normal((1, total, 2 * 2 + 16, 128), 73)
    idx = _normal((1, total, 1, 128), 74)
    q_rot = torch.empty((1, total, 16, 128), dtype=torch.bfloat16, device="cuda")
    pos = _i32(np.arange(total)[None])
    for lo, hi in ((0, 1000), (1000, n_ctx), (n_ctx, total)):  # two prefill chunks and the verify step's tokens
        s = slice(lo, hi)
        qsa.kv_append(d, x[:, s, 16:18], x[:, s, 18:], kc, vc, ks, vs, pt, pos[:, s].contiguous(), ws, rope=rope,
                      q=x[:, s, :16], q_out=q_rot[:, s])
    idx_keys = torch.zeros((1, 4 * d.max_blocks, 1, 128), dtype=torch.bfloat16, device="cuda")
    qsa.rope(rope, idx[:, :4 * d.max_blocks], pos[:, :4 * d.max_blocks].contiguous(), idx_keys)
    q_pos = pos[:, n_ctx:].contiguous()
    kcomp = torch.zeros((1, d.max_blocks, 1, 128), dtype=torch.bfloat16, device="cuda")
    q, q_idx = q_rot[:, n_ctx:].contiguous(), idx[:, n_ctx:].contiguous()
    sparse, dense = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty((1, n_q, 16), device="cuda")
    qsa.compress_keys(d, idx_keys, q_pos, kcomp, ws)
    for _ in range(2):
        qsa.decode(d, q_idx, kcomp, q, kc, vc, ks, vs, pt, q_pos, sparse, ws)
        qsa.paged_attn(d, q, kc, vc, ks, vs, pt, q_pos, dense, ws, lse=lse)
        _ok(qsa, ws)
        _compare_attn((d, q, kc, vc, ks, vs, pt, q_pos, dense, ws), lse)
        _compare_attn((d, q, kc, vc, ks, vs, pt, q_pos, sparse, ws), lse)
    # what was written reads back
    ko, vo = (torch.empty((1, total, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qsa.kv_gather(d, kc, vc, ks, vs, pt, pos, ko, vo, ws)
    _ok(qsa, ws)
    if kv == "bf16":
        assert torch.equal(vo, x[:, :, 18:])
        want = torch.empty_like(ko)
        qsa.rope(rope, x[:, :, 16:18], pos, want)
        assert torch.equal(ko, want)
    else:
        v = x[:, :, 18:].float()
        assert torch.all((vo.float() - v).abs() <= 2.0 ** -4 * v.abs() + 2.0 ** -10 * vs.max() + 2.0 ** -8 * v.abs())


@pytest.mark.parametrize("how", ["rope", "append", "attention"])
def test_what_follows_reads_what_was_written(qsa, how):
    # qsa_sparse_attn_rows loads its queries before it waits for the kernel in
    # front of it: whatever of this library wrote them, in calls back to back,
    # they are there
    B, n_q, n = 32, 4, 3000
    per = -(-n // 64)
    d = qsa.make_dims(B, n_q, n // 4, per, B * per)
    kc, vc, _, _ = R.make_cache(B * per, 2, 64, 128, "bf16", 81)
    pt = torch.randperm(B * per, device="cuda").to(torch.int32).view(B, per)
    pos = _i32(np.tile(np.arange(n - n_q, n), (B, 1)))
    sel = torch.full((B, n_q, d.width), -1, dtype=torch.int32, device="cuda")
    sel[:, :, :512] = torch.arange(512, dtype=torch.int32, device="cuda") * 5  # below every query's position
    ws = torch.zeros(max(qsa.workspace_size(d), qsa.kv_workspace_size(d)), dtype=torch.uint8, device="cuda")
    rows = torch.empty_like(sel)
    qsa.resolve(d, sel, pos, pt, rows, ws)
    rope = qsa.make_rope(128)
    xs = [_normal((B, n_q, 20, 128), 82 + i) for i in range(3)]
    ws2 = qsa.make_kv_workspace(d)

    def make_q(x, q):
        if how == "rope":
            qsa.rope(rope, x[:, :, :16], pos, q)
        elif how == "append":
            qsa.kv_append(d, x[:, :, 16:18], x[:, :, 18:], kc, vc, None, None, pt, pos, ws2, rope=rope,
                          q=x[:, :, :16], q_out=q)
        else:
            qsa.paged_attn(d, x[:, :, :16].contiguous(), kc, vc, None, None, pt, pos, q, ws2)

    def calls():
        for i in range(12):
            make_q(xs[i % 3], qs[i])
            qsa.sparse_attn_rows(d, qs[i], kc, vc, None, None, rows, outs[i], ws)

    qs, outs = ([torch.full((B, n_q, 16, 128), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(12)]
                for _ in range(2))
    want = []
    for i in range(12):
        make_q(xs[i % 3], qs[i])
        torch.cuda.synchronize()
        qsa.sparse_attn_rows(d, qs[i], kc, vc, None, None, rows, outs[i], ws)
        torch.cuda.synchronize()
        want.append(outs[i].clone())
        assert not torch.isnan(want[i]).any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for go in (calls, graph.replay, graph.replay):
        for t in qs + outs:
            t.fill_(math.nan)
        go()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    _ok(qsa, ws)
    _ok(qsa, ws2)


@pytest.mark.parametrize("B", [1, 32])
def test_rows_attention_reads_queries_behind_its_wait(qsa, B):
    # qsa_sparse_attn_rows behind a kernel that lets its successor start at once
    # and then writes the queries: qsa_resolve is one, its cache rows 16,128 ..
    # 16,639 taken as the bits of BF16 queries (0.5 to 3.1 in every second place).
    # B 1: the cluster form, 32: equal shares of the stream
    n_q, n, ps = 4, 600, 64
    per = -(-n // ps)
    d = qsa.make_dims(B, n_q, n // 4, per, B * per)
    kc, vc, _, _ = R.make_cache(B * per, 2, ps, 128, "bf16", 91)
    pt = torch.randperm(B * per, device="cuda").to(torch.int32).view(B, per)
    pos = _i32(np.tile(np.arange(n - n_q, n), (B, 1)))
    g = torch.Generator("cuda").manual_seed(92)
    sel = torch.full((B, n_q, d.width), -1, dtype=torch.int32, device="cuda")
    sel[:, :, :512] = torch.randint(0, n - n_q, (B, n_q, 512), generator=g, device="cuda", dtype=torch.int32)
    ws = torch.zeros(qsa.workspace_size(d), dtype=torch.uint8, device="cuda")
    rows = torch.empty_like(sel)
    qsa.resolve(d, sel, pos, pt, rows, ws)
    # the kernel that writes the queries
    d2 = qsa.make_dims(B, n_q, 64, 4, 130)
    pt2 = _i32([[126, 127, 128, 129]] * B)
    pos2 = torch.full((B, n_q), 255, dtype=torch.int32, device="cuda")
    sel2 = [torch.randint(0, 256, sel.shape, generator=g, device="cuda", dtype=torch.int32) for _ in range(3)]
    ws2 = torch.zeros(qsa.workspace_size(d2), dtype=torch.uint8, device="cuda")
    made = [torch.empty_like(sel) for _ in range(12)]
    qs = [m.view(-1)[:B * n_q * 1024].view(torch.bfloat16).view(B, n_q, 16, 128) for m in made]
    outs = [torch.empty((B, n_q, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(12)]

    def calls(sync=False):
        for i in range(12):
            qsa.resolve(d2, sel2[i % 3], pos2, pt2, made[i], ws2)
            if sync:
                torch.cuda.synchronize()
            qsa.sparse_attn_rows(d, qs[i], kc, vc, None, None, rows, outs[i], ws)

    calls(sync=True)
    want = [o.clone() for o in outs]
    assert torch.isfinite(want[0]).all() and not torch.equal(want[0], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for go in (calls, graph.replay, graph.replay):
        for m, o in zip(made, outs):
            m.fill_(-1)  # NaN
            o.fill_(math.nan)
        go()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    _ok(qsa, ws)
    _ok(qsa, ws2)


def test_calls_without_the_fast_path(qsa, monkeypatch):
    # the binding's own checks make the same calls
    ctx, n_q, ps = [300, 64], 2, 64
    args, lse = _attn_case(qsa, ctx, n_q, 16, 2, 128, ps, "fp8")
    d, q, kc, vc, ks, vs, table, pos, out, ws = args
    x, rope = _normal((2, n_q, 20, 128), 95), qsa.make_rope(128)

    def calls():
        kc2, vc2, q_out, y = kc.clone(), vc.clone(), torch.empty_like(q), torch.empty_like(q)
        ko, vo = (torch.empty((2, n_q, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        o, l = torch.empty_like(out), torch.empty_like(lse)
        qsa.kv_append(d, x[:, :, 16:18], x[:, :, 18:], kc2, vc2, ks, vs, table, pos, ws, rope=rope, q=x[:, :, :16],
                      q_out=q_out)
        qsa.kv_gather(d, kc2, vc2, ks, vs, table, pos, ko, vo, ws)
        qsa.rope(rope, x[:, :, :16], pos, y, inverse=True, stream=torch.cuda.current_stream())
        qsa.paged_attn(d, q_out, kc2, vc2, ks, vs, table, pos, o, ws, lse=l, window=100)
        _ok(qsa, ws)
        return kc2, vc2, q_out, y, ko, vo, o, l

    want = calls()
    assert qsa._fast is not qsa._NoFast
    monkeypatch.setattr(qsa, "_fast", qsa._NoFast)
    assert all(torch.equal(a, b) for a, b in zip(calls(), want))


@pytest.mark.parametrize("kv,D,n_q", [("bf16", 128, 1), ("fp8", 64, 4), ("bf16", 256, 2), ("fp8", 128, 4)])
def test_attn_wait_runs_out_and_reports_a_timeout(qsa, kv, D, n_q):
    # Failure detection without a fault: the test hook's copies of K bring half
    # of the bytes that the kernel waits for, so every CTA's wait for its first
    # tile runs out (about a second). The timeout is reported, every role of the
    # kernel ends and its tensor memory is free: the next calls, which need all
    # of it again, are complete.
    import time

    args, lse = _attn_case(qsa, [1500, 70, 0, 300], n_q, 16, 2, D, 64, kv)
    out, ws = args[8], args[9]
    want, want_lse = out.clone(), lse.clone()
    torch.cuda.synchronize()
    t0 = time.time()
    qsa.test_paged_attn_timeout(*args, lse=lse)
    torch.cuda.synchronize()
    waited = time.time() - t0
    st, info = qsa.check_errors(ws)
    assert st == qsa.ERR_TIMEOUT and info[0] == 5, info
    assert 0.2 < waited < 30, waited
    for _ in range(3):
        out.fill_(7.0)
        lse.fill_(7.0)
        qsa.paged_attn(*args, lse=lse)
        _ok(qsa, ws)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
