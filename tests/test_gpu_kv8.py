"""8-bit K/V cache on the GPU: writer, attention and eviction against the fp64
oracle, at the sizes, masks and layouts where they can go wrong."""

import math

import numpy as np
import pytest
import torch

import looped_transformer_latent_b200 as L
from oracle import kv8

pytestmark = pytest.mark.gpu
DT = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _codes(t):
    """Stored codes as the values they are, fp64 on the host."""
    return t.to(torch.float64).cpu().numpy()


def _f64(t):
    return t.double().cpu().numpy()


def _randn(g, *shape):
    x = torch.randn(*shape, generator=g)
    return x * (1 + 3 * (torch.rand(shape[-1], generator=g) > 0.9))


class Cache:
    """A cache of random tokens, quantised by the oracle; rows past each length hold the worst codes and scales."""

    def __init__(self, seed, B, H, d, block, cap, code, lens):
        g = torch.Generator().manual_seed(seed)
        self.block, self.lens, self.code = block, lens, code
        fill = torch.full((B, H, cap, d), 0x7F, dtype=torch.uint8)
        self.values = {}
        for n in ("k", "v"):
            codes, scales = fill.clone().view(DT[code]), torch.full((B, H, cap // block), math.nan)
            self.values[n] = []
            for b in range(B):
                per = []
                for h in range(H):
                    c, s = kv8.write(_randn(g, lens[b], d).numpy(), block, code)
                    codes[b, h, :lens[b]] = torch.from_numpy(c).float().to(DT[code])
                    scales[b, h, :len(s)] = torch.from_numpy(s)
                    per.append(kv8.values(c, s, block))
                self.values[n].append(np.stack(per))
            setattr(self, n + "8", codes.cuda())
            setattr(self, n + "_scale", scales.cuda())

    def args(self):
        return dict(k8=self.k8, v8=self.v8, k_scale=self.k_scale, v_scale=self.v_scale)


# ------------------------------------------------------------------- write --
WRITE = [  # B, H, d, block, n, code, io
    (1, 1, 16, 16, 1, "i8", "bf16"), (2, 3, 64, 32, 64, "e4m3", "bf16"), (2, 2, 96, 64, 129, "i8", "f32"),
    (1, 2, 128, 128, 300, "e4m3", "f32"), (3, 1, 256, 16, 47, "i8", "bf16"), (1, 5, 80, 256, 257, "e4m3", "bf16"),
    (2, 2, 48, 32, 31, "e4m3", "f32"), (1, 1, 112, 64, 640, "i8", "bf16"), (1, 3, 240, 256, 256, "i8", "f32"),
]


@pytest.mark.parametrize("B,H,d,block,n,code,io", WRITE)
def test_write_gives_the_oracles_codes(B, H, d, block, n, code, io):
    g = torch.Generator().manual_seed(n)
    k, v = (_randn(g, B, n, H, d).to(IO[io]) for _ in range(2))
    cap = -(-n // block) * block + block
    k8, v8 = (torch.full((B, H, cap, d), 7, device="cuda").to(DT[code]) for _ in range(2))
    ks, vs = (torch.full((B, H, cap // block), 5.0, device="cuda") for _ in range(2))
    L.lla_kv8_write(k=k.cuda(), v=v.cuda(), k8=k8, v8=v8, k_scale=ks, v_scale=vs, row0=block)
    for x, x8, xs in ((k, k8, ks), (v, v8, vs)):
        got, scales = _codes(x8), xs.cpu().numpy()
        for b in range(B):
            for h in range(H):
                c, s = kv8.write(x[b, :, h].float().numpy(), block, code)
                assert np.array_equal(got[b, h, block:block + n], c)
                assert np.array_equal(scales[b, h, 1:1 + len(s)], s)
                assert np.all(got[b, h, :block] == 7) and np.all(got[b, h, block + n:] == 7)   # left as they were
                assert scales[b, h, 0] == 5


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_write_from_a_ring_ragged_and_misfits(code, io):
    B, H, d, block, rows = 6, 2, 64, 16, 48
    g = torch.Generator().manual_seed(3)
    k, v = (_randn(g, B, rows, H, d).to(IO[io]) for _ in range(2))
    k8, v8 = (torch.zeros(B, H, 64, d, device="cuda").to(DT[code]) for _ in range(2))
    ks, vs = (torch.zeros(B, H, 4, device="cuda") for _ in range(2))
    n, src0, row0 = [16, 33, 0, 20, 20, 32], [40, 1000, 5, 0, 7, -3], [0, 16, 16, 8, 48, 32]
    L.lla_kv8_write(k=k.cuda(), v=v.cuda(), k8=k8, v8=v8, k_scale=ks, v_scale=vs, n=_i32(n), max_n=48, src0=_i32(src0),
                    row0=_i32(row0), ring=True)
    want, scales = np.zeros((B, H, 64, d)), np.zeros((B, H, 4), dtype=np.float32)
    for b in range(B):
        if row0[b] % block or row0[b] + n[b] > 64:
            continue            # sequences 3 (row0 inside a block) and 4 (past the end) are left as they were
        at = [(src0[b] + i) % rows for i in range(n[b])]
        for h in range(H):
            c, s = kv8.write(k[b, at, h].float().numpy().reshape(-1, d), block, code)
            want[b, h, row0[b]:row0[b] + n[b]] = c
            scales[b, h, row0[b] // block:row0[b] // block + len(s)] = s
    assert np.array_equal(_codes(k8), want) and np.array_equal(ks.cpu().numpy(), scales)


def test_write_plain_rows_that_do_not_fit_are_left():
    x = torch.ones(3, 32, 1, 16, device="cuda")
    k8 = torch.zeros(3, 1, 32, 16, dtype=torch.int8, device="cuda")
    s = torch.zeros(3, 1, 2, device="cuda")
    L.lla_kv8_write(k=x, v=x, k8=k8, v8=k8.clone(), k_scale=s, v_scale=s.clone(), n=_i32([16, 99, -4]),
                    src0=_i32([17, 0, 0]), max_n=32)
    assert not k8[0].any() and not k8[2].any()      # 17 + 16 rows of 32; a negative count is none
    assert (k8[1] == 127).all()                     # 99 is clamped to max_n


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_write_zero_tiny_and_non_finite_blocks(code, bad):
    x = torch.zeros(1, 96, 2, 32)
    x[0, 40, 0, 3] = bad
    x[0, 64:, 1] = torch.randn(32, 32, generator=torch.Generator().manual_seed(1)) * 1e-42    # subnormal
    x[0, 64:, 0] = 3e38
    k8 = torch.full((1, 2, 96, 32), 3, device="cuda").to(DT[code])
    s = torch.full((1, 2, 3), 9.0, device="cuda")
    L.lla_kv8_write(k=x.cuda(), v=x.cuda(), k8=k8, v8=k8.clone(), k_scale=s, v_scale=s.clone())
    for h in range(2):
        c, sc = kv8.write(x[0, :, h].numpy(), 32, code)
        assert np.array_equal(_codes(k8)[0, h], c)
        assert np.array_equal(s.cpu().numpy()[0, h], sc, equal_nan=True)


def test_write_reads_and_writes_strided_views():
    g = torch.Generator().manual_seed(5)
    ring = torch.randn(2, 3, 32, 4, 32, generator=g).cuda()          # [B, T, rows, H, d]
    k, v = ring[:, 1, :, :2], ring[:, 2, :, 2:]
    k8 = torch.zeros(3, 2, 2, 64, 32, dtype=torch.int8, device="cuda")   # [T, H, B, ...]
    s = torch.zeros(3, 2, 2, 4, device="cuda")
    c8, cs = k8[1].transpose(0, 1), s[1].transpose(0, 1)
    d8, ds = k8[2].transpose(0, 1), s[2].transpose(0, 1)
    L.lla_kv8_write(k=k, v=v, k8=c8, v8=d8, k_scale=cs, v_scale=ds, row0=32)
    for x, x8, xs in ((k, c8, cs), (v, d8, ds)):
        for b in range(2):
            for h in range(2):
                c, sc = kv8.write(x[b, :, h].cpu().numpy(), 16, "i8")
                assert np.array_equal(_codes(x8)[b, h, 32:], c) and np.array_equal(xs.cpu().numpy()[b, h, 2:], sc)
    assert not k8[0].any()


# --------------------------------------------------------------- attention --
def _run_attn(c, q, win=None, ctx=None, tail=None, weights=None, scale=0.0, **kw):
    out = torch.full_like(q, 77.0)
    L.lla_kv8_attn(q=q, out=out, lens=_i32(c.lens), weights=weights, scale=scale, **c.args(),
                   **(dict(win_k=win[0], win_v=win[1], ctx=_i32(ctx), tail=_i32(tail)) if win else {}), **kw)
    return out


def _check(c, q, out, win=None, ctx=None, tail=None, weights=None, before=None, scale=0.0):
    """Against the oracle, within bounds from the formats: delta bounds the error of a score (a query as two f16 terms
    is off by 2^-22, d products are summed in fp32), a weight is off by twice that and by the sum over n tokens, and
    16-bit calls round probabilities to f16 (2^-11 each, and the exact ones no coarser) and the output to bf16."""
    B, nq, HG, d = q.shape
    H = c.k8.shape[1]
    G = HG // H
    half = q.dtype == torch.bfloat16
    q64, o64 = _f64(q).reshape(B, nq, H, G, d), _f64(out).reshape(B, nq, H, G, d)
    sc = scale or 1 / math.sqrt(d)
    for b in range(B):
        k, v = c.values["k"][b], c.values["v"][b]
        if win:
            wk, wv = (kv8.ring_rows(_f64(x[b]), ctx[b], tail[b]).reshape(tail[b], H, d) for x in win)
        else:
            wk = wv = np.zeros((0, H, d))
        ref, w = kv8.attn(q64[b], k, v, wk, wv, scale)
        n = k.shape[1] + len(wk)
        kk, vv = np.concatenate([k, wk.transpose(1, 0, 2)], 1), np.concatenate([v, wv.transpose(1, 0, 2)], 1)
        if n == 0:
            assert not o64[b].any()
            continue
        top = sc * np.einsum("phgd,hjd->phgj", np.abs(q64[b]), np.abs(kk)).max()
        delta = top * (2.0 ** -22 + (d + 4) * 2.0 ** -24)
        rel = 2 * delta + 2.0 ** -20 + n * 2.0 ** -23
        tol = np.abs(vv).max() * (rel + (2.0 ** -10 if half else 0)) + (2.0 ** -8 * np.abs(ref) if half else 0)
        assert np.all(np.abs(o64[b] - ref) <= tol), np.abs(o64[b] - ref).max()
        if weights is not None:
            got, was = _f64(weights[b]), _f64(before[b])
            m = k.shape[1]
            assert np.all(np.abs(got[:, :m] - was[:, :m] - w) <= rel * w + 2.0 ** -23 * (was[:, :m] + w) + 1e-30)
            assert np.array_equal(got[:, m:], was[:, m:])       # past the length: left as they were


ATTN = [  # B, H, G, nq, d, block, lens, code, io, Wcap, tails, win dtype
    (1, 1, 1, 1, 16, 16, [1], "i8", "bf16", 0, None, None),
    (2, 2, 1, 1, 64, 32, [0, 31], "e4m3", "bf16", 8, [0, 3], "bf16"),          # one sequence sees nothing
    (3, 2, 1, 1, 128, 64, [200, 1, 64], "i8", "bf16", 64, [64, 1, 17], "bf16"),
    (2, 1, 4, 1, 128, 64, [333, 65], "e4m3", "bf16", 32, [7, 32], "bf16"),
    (1, 2, 8, 1, 96, 32, [129], "i8", "f32", 16, [16], "f32"),
    (2, 3, 2, 1, 80, 16, [47, 17], "e4m3", "f32", 5, [5, 0], "bf16"),
    (1, 1, 32, 1, 96, 64, [300], "i8", "bf16", 0, None, None),
    (1, 2, 1, 5, 64, 32, [100], "i8", "bf16", 16, [9], "bf16"),                # several positions
    (2, 1, 3, 17, 128, 64, [70, 130], "e4m3", "bf16", 64, [17, 40], "bf16"),
    (1, 1, 2, 64, 96, 32, [97], "i8", "f32", 64, [64], "f32"),
    (2, 2, 1, 33, 128, 64, [0, 190], "e4m3", "f32", 64, [20, 33], "bf16"),     # early queries see nothing
    (1, 1, 1, 3, 256, 128, [257], "i8", "bf16", 4, [4], "f32"),
    (1, 2, 5, 1, 240, 256, [500], "e4m3", "bf16", 3, [2], "bf16"),
    (1, 1, 9, 1, 32, 16, [1000], "i8", "f32", 0, None, None),
    (4, 1, 1, 1, 48, 16, [16, 15, 640, 2], "i8", "bf16", 33, [33, 1, 2, 0], "bf16"),
    (1, 1, 64, 2, 64, 64, [65], "e4m3", "bf16", 4, [3], "bf16"),
    (1, 4, 1, 1, 128, 128, [2500], "i8", "f32", 129, [129], "bf16"),
    (1, 2, 1, 130, 128, 64, [321], "e4m3", "bf16", 192, [150], "bf16"),
    (1, 1, 4, 70, 64, 32, [77], "i8", "bf16", 128, [128], "f32"),
]


def _inputs(case, seed=0):
    B, H, G, nq, d, block, lens, code, io, wcap, tails, wdt = case
    cap = -(-max(max(lens), 1) // block) * block + block
    c = Cache(seed, B, H, d, block, cap, code, lens)
    g = torch.Generator().manual_seed(seed + 1)
    q = (2 * torch.randn(B, nq, H * G, d, generator=g)).to(IO[io]).cuda()
    win = ctx = None
    if wcap:
        win = [_randn(g, B, wcap, H, d).to(IO[wdt]) for _ in range(2)]
        ctx = [lens[b] + tails[b] + 11 * b for b in range(B)]     # as after an eviction: ctx is not len + tail
        for b in range(B):      # slots that no query may see hold what must not be used
            dead = [j % wcap for j in range(ctx[b], ctx[b] - tails[b] + wcap)]
            for x in win:
                x[b, dead] = math.nan
        win = [x.cuda() for x in win]
    w = torch.rand(B, H, cap, generator=g).cuda()
    return c, q, win, ctx, tails, w


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_attention_against_the_oracle(case):
    c, q, win, ctx, tails, w = _inputs(case)
    before = w.clone()
    plain = _run_attn(c, q, win, ctx, tails)
    out = _run_attn(c, q, win, ctx, tails, weights=w)
    _check(c, q, plain, win, ctx, tails)                 # with and without the accumulator the splits may differ
    _check(c, q, out, win, ctx, tails, w, before)
    assert torch.equal(_run_attn(c, q, win, ctx, tails), plain)
    again, w2 = _run_attn(c, q, win, ctx, tails, weights=(w2 := before.clone())), w2
    assert torch.equal(again, out) and torch.equal(w2, w)    # deterministic


def test_attention_scale_ints_strides_and_shared_rows():
    B, H, G, d, block = 2, 2, 2, 64, 32
    c = Cache(9, B, H, d, block, 128, "i8", [96, 96])
    g = torch.Generator().manual_seed(2)
    big = torch.randn(B, 3, 3, H * G, d, generator=g).cuda()
    q, out = big[:, 1, ::2], torch.zeros(B, 4, H * G, d, device="cuda")[:, 1:3]
    ring = torch.randn(B, 2, 8, 3, d, generator=g).to(torch.bfloat16).cuda()
    win = [ring[:, 0, :, :2], ring[:, 1, :, 1:]]
    w = torch.zeros(H, B, 256, device="cuda").transpose(0, 1)[..., :128]
    L.lla_kv8_attn(q=q, out=out, lens=96, scale=0.07, weights=w, win_k=win[0], win_v=win[1], ctx=101, tail=5, **c.args())
    _check(c, q, out, win, [101] * 2, [5] * 2, w, torch.zeros_like(w), scale=0.07)
    # one prefix read by both sequences: sequence 0's rows through a zero stride
    one = {n: t[:1].expand(2, *t.shape[1:]) for n, t in c.args().items()}
    same = torch.zeros_like(q)
    L.lla_kv8_attn(q=q, out=same, lens=96, scale=0.07, **one)
    c.values = {n: [x[0], x[0]] for n, x in c.values.items()}
    _check(c, q, same, scale=0.07)


def test_attention_large_logits_and_far_apart_scales():
    B, H, d, block = 1, 1, 64, 16
    c = Cache(4, B, H, d, block, 160, "i8", [150])
    f = torch.tensor([2.0 ** e for e in (0, -40, 5, -120, 30, 2, -3, 60, 1, -10)], device="cuda")
    c.v_scale *= f
    c.values["v"][0] = c.values["v"][0] * np.repeat(f.cpu().numpy().astype(np.float64), 16)[None, :150, None]
    q = (20 * torch.randn(1, 1, 3, d, generator=torch.Generator().manual_seed(0))).cuda()
    _check(c, q, _run_attn(c, q))
    z = torch.zeros_like(q)
    _check(c, z, _run_attn(c, z))                       # all logits equal
    tiny = (q * 1e-30).to(torch.bfloat16)
    _check(c, tiny, _run_attn(c, tiny))
    huge = (q * 1e4).to(torch.bfloat16)                 # beyond the range of f16; the bound on the scores says nothing
    k64, v64 = c.values["k"][0], c.values["v"][0]
    got = _f64(_run_attn(c, huge))[0, 0]
    for r in range(3):
        s = k64[0] @ _f64(huge)[0, 0, r]
        top, second = np.sort(s)[::-1][:2]
        if (top - second) / 8 > 1e3:
            assert np.all(np.abs(got[r] - v64[0, s.argmax()]) <= 2.0 ** -7 * np.abs(v64[0, s.argmax()]))


@pytest.mark.parametrize("d", [48, 96, 128])
@pytest.mark.parametrize("G", [33, 64, 100, 160])
def test_attention_of_many_rows_with_far_apart_scales(G, d):
    """Rows beyond 32 go to the tcgen05 kernel; scales of values 2^-40 to 2^30 apart, one block zero, several splits."""
    code = "i8" if G % 2 else "e4m3"
    c = Cache(G, 2, 1, d, 32, 1312, code, [1300, 70])
    w = torch.zeros(2, 1, 1312, device="cuda")
    q = (2 * torch.randn(2, 1, G, d, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).cuda()
    _check(c, q, _run_attn(c, q, weights=w), weights=w, before=torch.zeros_like(w))
    f = torch.tensor([2.0 ** e for e in (0, -40, 5, -20, 30, 2, -3, 0, 1, -10)] * 5, device="cuda")[:41]
    f[3] = 0
    c.v_scale *= f
    f = f.cpu().double().numpy()
    c.values["v"] = [v * f[np.arange(v.shape[1]) // 32][None, :, None] for v in c.values["v"]]
    _check(c, q, _run_attn(c, q))
    # logits so far apart that one token has all the weight, wherever its block's scale lies
    big = (100 * q.float()).to(torch.bfloat16)
    got = _f64(_run_attn(c, big))
    for b in range(2):
        k, v = c.values["k"][b][0], c.values["v"][b][0]
        for r in range(G):
            s = k @ _f64(big)[b, 0, r] / math.sqrt(d)
            top, second = np.sort(s)[::-1][:2]
            # the others' shares are at most exp(second - top) each, on values up to the largest of all
            rest = len(s) * math.exp(second - top) * np.abs(v).max()
            if top - second > 60:
                want = v[s.argmax()]
                assert np.all(np.abs(got[b, 0, r] - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -10 * np.abs(want).max() + 2 * rest)


@pytest.mark.parametrize("G", [1, 40])
def test_attention_keeps_what_a_query_does_not_see_out_of_it(G):
    """A later position's value or key that is no number reaches that position's queries only."""
    for wdt in ("bf16", "f32"):
        c = Cache(3, 1, 2, 64, 32, 96, "i8", [70])
        g = torch.Generator().manual_seed(1)
        q = torch.randn(1, 3, 2 * G, 64, generator=g).to(torch.bfloat16).cuda()
        win = [torch.randn(1, 8, 2, 64, generator=g).to(IO[wdt]).cuda() for _ in range(2)]
        clean = _run_attn(c, q, win, [90], [6])
        for ring, bad in ((1, math.inf), (1, math.nan), (0, math.nan)):
            dirty = [x.clone() for x in win]
            dirty[ring][0, 89 % 8, 1, 5] = bad           # the last position, head 1
            out = _run_attn(c, q, dirty, [90], [6])
            assert torch.equal(out[:, :2], clean[:, :2]) and torch.equal(out[:, 2, :G], clean[:, 2, :G])
            assert not torch.isfinite(out[:, 2, G:]).all(-1).any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention_of_more_heads_and_rows_than_a_grid_holds(io):
    H, G, d = 30000, 300, 16                             # 3 or more row tiles of 30000 heads
    g = torch.Generator(device="cuda").manual_seed(0)
    k8, v8 = (torch.randint(-127, 128, (1, H, 16, d), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    s = torch.full((1, H, 1), 0.01, device="cuda")
    q = torch.randn(1, 1, H * G, d, generator=g, device="cuda").to(IO[io])
    out = torch.zeros_like(q)
    L.lla_kv8_attn(q=q, out=out, lens=5, k8=k8, v8=v8, k_scale=s, v_scale=s)
    for h0 in range(0, H, 10000):
        at = slice(h0, h0 + 10000)
        k, v = (x[0, at, :5].double() * 0.01 for x in (k8, v8))
        a = torch.softmax(q[0, 0].view(H, G, d)[at].double() @ k.transpose(1, 2) / math.sqrt(d), -1)
        # values up to 1.27; the bound on the rounding of a weight as above, and the output's own
        err = (out[0, 0].view(H, G, d)[at].double() - a @ v).abs().max().item()
        assert err <= 1.27 * ((2.0 ** -10 + 2.0 ** -8) if io == "bf16" else 2.0 ** -16)


def test_weights_of_more_rows_than_one_pass_holds():
    n, d, G = 1 << 20, 16, 96                            # scores of 64 rows fill a pass: two passes
    g = torch.Generator(device="cuda").manual_seed(0)
    k8, v8 = (torch.randint(-127, 128, (1, 1, n, d), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand(1, 1, n // 256, generator=g, device="cuda") * 0.01 + 0.01 for _ in range(2))
    q = torch.randn(1, 1, G, d, generator=g, device="cuda").to(torch.bfloat16)
    out, w = torch.empty_like(q), torch.zeros(1, 1, n, device="cuda")
    m = n - 77
    L.lla_kv8_attn(q=q, out=out, lens=m, k8=k8, v8=v8, k_scale=ks, v_scale=vs, weights=w)
    k, v = (x[0, 0, :m].double() * s[0, 0].double().repeat_interleave(256)[:m, None] for x, s in ((k8, ks), (v8, vs)))
    a = torch.softmax(q[0, 0].double() @ k.T / math.sqrt(d), -1)
    ref = a @ v
    top = (q[0, 0].double().abs() @ k.abs().T / math.sqrt(d)).max().item()
    rel = 2 * top * (2.0 ** -22 + (d + 4) * 2.0 ** -24) + 2.0 ** -20 + 2.0 ** -24 * 4096   # longest run of one fp32 sum
    assert ((out[0, 0].double() - ref).abs() <= v.abs().max() * (rel + 2.0 ** -10) + 2.0 ** -8 * ref.abs()).all()
    want = a.sum(0)
    assert ((w[0, 0, :m].double() - want).abs() <= (rel + 2.0 ** -20) * want + 1e-30).all() and not w[0, 0, m:].any()


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_attention_of_a_block_of_nan_is_nan_in_its_head_only(code):
    c = Cache(4, 1, 2, 64, 16, 64, code, [50])
    for part in ("k_scale", "v_scale"):
        was = getattr(c, part).clone()
        getattr(c, part)[0, 1, 2] = math.nan
        q = torch.randn(1, 2, 4, 64, generator=torch.Generator().manual_seed(0)).cuda()
        out = _run_attn(c, q)
        assert torch.isnan(out[:, :, 2:]).all() and not torch.isnan(out[:, :, :2]).any()
        getattr(c, part).copy_(was)


def test_attention_offsets_past_32_bits():
    H, d, block, cap = 3, 128, 64, 9 << 20              # 1.2 GB of codes for each head
    k8 = torch.empty(1, H, cap, d, dtype=torch.int8, device="cuda")
    s = torch.zeros(1, H, cap // block, device="cuda")
    small = Cache(6, 1, H, d, block, 128, "i8", [100])
    k8[:, :, :128], s[:, :, :2] = small.k8, small.k_scale
    # the last block of the last head through a view that starts past 2^31 bytes
    view = k8[:, :, cap - 128:]
    view.copy_(small.k8)
    args = dict(k8=view, v8=view, k_scale=small.k_scale, v_scale=small.k_scale)
    q = torch.randn(1, 1, H, d, generator=torch.Generator().manual_seed(0)).cuda()
    out, ref = torch.empty_like(q), torch.empty_like(q)
    L.lla_kv8_attn(q=q, out=out, lens=100, **args)
    L.lla_kv8_attn(q=q, out=ref, lens=100, k8=small.k8, v8=small.k8, k_scale=small.k_scale, v_scale=small.k_scale)
    assert torch.equal(out, ref)
    del k8, view, args
    # one long head: tokens on both sides of 2^31 bytes
    cap = (1 << 24) + 4096
    k8 = torch.zeros(1, 1, cap, d, dtype=torch.int8, device="cuda")
    s = torch.full((1, 1, cap // block), 0.05, device="cuda")
    k8[0, 0, cap - 100] = 127
    v8 = torch.zeros_like(k8)
    v8[0, 0, cap - 100:cap - 99] = torch.arange(d, device="cuda").to(torch.int8)
    q = torch.full((1, 1, 1, d), 4.0, device="cuda")    # that token's logit is 286, every other's 0
    out = torch.empty_like(q)
    w = torch.zeros(1, 1, cap, device="cuda")
    L.lla_kv8_attn(q=q, out=out, lens=cap - 3, k8=k8, v8=v8, k_scale=s, v_scale=s, weights=w)
    assert torch.allclose(out[0, 0, 0], 0.05 * torch.arange(d, device="cuda"), rtol=1e-6, atol=0)
    # a logit of 286 from d products summed in fp32 is off by at most 286 (d + 4) 2^-24 = 2.3e-3 each time it is formed
    assert abs(w[0, 0, cap - 100].item() - 1) <= 2 * 286 * (d + 4) * 2.0 ** -24
    assert w.count_nonzero() == 1


def test_attention_in_graphs_that_share_a_workspace_and_on_other_streams():
    case = (3, 2, 2, 1, 64, 32, [90, 40, 64], "i8", "bf16", 16, [5, 9, 16], "bf16")
    c, q, win, ctx, tails, w = _inputs(case)
    c2, q2, _, _, _, w2 = _inputs(case, seed=50)
    lens, tail, ctx_t = _i32(c.lens), _i32(tails), _i32(ctx)
    out, out2 = torch.zeros_like(q), torch.zeros_like(q)
    a = dict(q=q, out=out, lens=lens, win_k=win[0], win_v=win[1], ctx=ctx_t, tail=tail, weights=w, **c.args())
    a2 = dict(q=q2, out=out2, lens=lens, weights=w2, **c2.args())
    before, before2 = w.clone(), w2.clone()
    ws = torch.empty(max(L.lla_kv8_attn_workspace_bytes(**a), L.lla_kv8_attn_workspace_bytes(**a2)), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.lla_kv8_attn(workspace=ws, stream=side, **a)
    L.lla_kv8_attn(workspace=ws, stream=side, **a2)
    torch.cuda.synchronize()
    _check(c, q, out, win, ctx, tails, w, before)
    _check(c2, q2, out2, weights=w2, before=before2)
    graphs = []
    for args in (a, a2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.lla_kv8_attn(workspace=ws, **args)
        graphs.append(g)
    w.copy_(before)
    w2.copy_(before2)
    # lengths are read when the graph runs
    c.lens, c2.lens = [90, 1, 0], [90, 1, 0]
    lens.copy_(_i32(c.lens))
    for x in (c, c2):
        x.values = {n: [v[b][:, :x.lens[b]] for b in range(3)] for n, v in x.values.items()}
    for _ in range(2):
        for g in graphs:
            out.zero_(), out2.zero_()
            w.copy_(before), w2.copy_(before2)
            for h in graphs:
                h.replay()
    torch.cuda.synchronize()
    _check(c, q, out, win, ctx, tails, w, before)
    _check(c2, q2, out2, weights=w2, before=before2)


# ---------------------------------------------------------------- eviction --
EVICT = [  # B, H, d, block, lens, keep, first, last, code
    (1, 1, 16, 16, [64], 2, 0, 1, "i8"), (2, 3, 64, 32, [320, 100], 4, 1, 2, "e4m3"),
    (3, 2, 128, 64, [0, 64, 1000], 5, 1, 1, "i8"), (2, 2, 96, 16, [481, 1], 7, 0, 3, "e4m3"),
    (1, 2, 256, 256, [2300], 3, 1, 2, "i8"), (1, 4, 48, 32, [900], 17, 2, 1, "i8"), (1, 1, 128, 16, [5003], 300, 1, 1, "i8"),
    (2, 1, 80, 16, [160, 161], 10, 4, 6, "e4m3"),
    (40, 4, 16, 16, [16 * (i % 9) + i % 17 + (i == 3) * 900 for i in range(40)], 3, 0, 1, "i8"),      # many heads
    (3, 60, 48, 32, [300, 0, 97], 2, 1, 1, "e4m3"),
]


def _weights(seed, B, H, cap, lens):
    w = torch.exp(2 * torch.randn(B, H, cap, generator=torch.Generator().manual_seed(seed)))
    for b in range(B):
        w[b, :, lens[b]:] = 0
    return w


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_eviction_against_the_oracle(case, inplace):
    B, H, d, block, lens, keep, first, last, code = case
    cap = -(-max(lens) // block) * block + block
    c = Cache(1, B, H, d, block, cap, code, lens)
    w = _weights(2, B, H, cap, lens)
    if max(lens) > 700:        # sums that are equal, and one that is no number
        w[-1, 0, :max(lens) // 2] = 0.25
        w[-1, 0, 3 * block + 1] = math.nan
    src = {n: t.cpu().view(torch.uint8).clone() if "8" in n else t.cpu().clone() for n, t in c.args().items()}
    wd = w.cuda()
    kept = torch.full((B, H, keep), 99, dtype=torch.int32, device="cuda")
    lens_t = _i32(lens)
    if inplace:
        to, t = None, dict(c.args(), weights=wd, lens=lens_t)
    else:
        dcap = keep * block + (block if lens[0] % 2 else 0)
        to = t = dict(k8=torch.full((B, H, dcap, d), 3, device="cuda").to(DT[code]),
                      v8=torch.full((B, H, dcap, d), 3, device="cuda").to(DT[code]),
                      k_scale=torch.full((B, H, dcap // block), 8.0, device="cuda"),
                      v_scale=torch.full((B, H, dcap // block), 8.0, device="cuda"),
                      weights=torch.full((B, H, dcap), 8.0, device="cuda"), lens=torch.zeros_like(lens_t))
    was = {n: t[n].cpu().view(torch.uint8).clone() if "8" in n else t[n].cpu().clone() for n in t}
    L.lla_kv8_evict(**c.args(), weights=wd, lens=lens_t, keep=keep, first=first, last=last, to=to, kept=kept)
    got = {n: t[n].cpu().view(torch.uint8) if "8" in n else t[n].cpu() for n in t}
    for b in range(B):
        nb = -(-lens[b] // block)
        new = lens[b] - max(0, nb - keep) * block
        assert got["lens"][b] == new
        for h in range(H):
            ids = kv8.choose(w[b, h].numpy(), lens[b], block, keep, first, last)
            assert kept[b, h].tolist() == ids + [-1] * (keep - len(ids))
            rows = [i * block + j for i in ids for j in range(block)][:new]
            for n in ("k8", "v8"):
                assert torch.equal(got[n][b, h, :new], src[n][b, h, rows])
                assert torch.equal(got[n][b, h, new:], was[n][b, h, new:])          # left as they were
            for n in ("k_scale", "v_scale"):
                assert torch.equal(got[n][b, h, :len(ids)], src[n][b, h, ids])
                assert torch.equal(got[n][b, h, len(ids):].nan_to_num(7.0), was[n][b, h, len(ids):].nan_to_num(7.0))
            assert torch.equal(got["weights"][b, h, :new].nan_to_num(-1.0), w[b, h, rows].nan_to_num(-1.0))
            end = min(lens[b], got["weights"].shape[2])
            assert not got["weights"][b, h, new:end].any()
            assert torch.equal(got["weights"][b, h, end:], was["weights"][b, h, end:])
    if not inplace:
        for n, x in c.args().items():
            assert torch.equal((x.cpu().view(torch.uint8) if "8" in n else x.cpu()).nan_to_num(7.0) if "8" not in n
                               else x.cpu().view(torch.uint8), src[n].nan_to_num(7.0) if "8" not in n else src[n])


def test_eviction_lengths_out_of_range_and_all_kept():
    c = Cache(1, 2, 1, 32, 16, 64, "i8", [64, 64])
    w = _weights(1, 2, 1, 64, [64, 64]).cuda()
    lens = _i32([1000, -5])
    was = c.k8.clone()
    L.lla_kv8_evict(**c.args(), weights=w, lens=lens, keep=4, first=1, last=1)
    assert lens.tolist() == [64, 0] and torch.equal(c.k8, was)


def test_eviction_in_a_graph():
    c = Cache(1, 2, 2, 64, 16, 160, "i8", [160, 100])
    w0 = _weights(1, 2, 2, 160, [160, 100])
    a = {n: t.clone() for n, t in c.args().items()}
    w, lens = w0.cuda(), _i32([160, 100])
    ws = torch.empty(L.lla_kv8_evict_workspace_bytes(**a, weights=w, lens=lens, keep=5, first=1, last=1),
                     dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lla_kv8_evict(**a, weights=w, lens=lens, keep=5, first=1, last=1, workspace=ws)
    assert lens.tolist() == [160, 100]
    g.replay()
    assert lens.tolist() == [80, 68]
    for b, n in enumerate((160, 100)):
        for h in range(2):
            ids = kv8.choose(w0[b, h].numpy(), n, 16, 5, 1, 1)
            rows = [i * 16 + j for i in ids for j in range(16)][:lens[b]]
            assert torch.equal(a["k8"][b, h, :lens[b]], c.k8[b, h, rows])


# ---------------------------------------------------------------- together --
@pytest.mark.parametrize("code,io", [("i8", "bf16"), ("e4m3", "f32")])
def test_a_serving_loop(code, io):
    """Decode steps over an exact ring; each full block of its oldest tokens is written to the cache, and a cache that
    is full is cut by the weights that the steps gathered."""
    B, H, G, d, block, wcap, cap, keep = 2, 2, 2, 64, 16, 48, 96, 4
    g = torch.Generator().manual_seed(8)
    ring = [torch.zeros(B, wcap, H, d, dtype=IO[io], device="cuda") for _ in range(2)]
    k8, v8 = (torch.zeros(B, H, cap, d, device="cuda").to(DT[code]) for _ in range(2))
    ks, vs = (torch.zeros(B, H, cap // block, device="cuda") for _ in range(2))
    w = torch.zeros(B, H, cap, device="cuda")
    lens, tail, ctx = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    cache = dict(k8=k8, v8=v8, k_scale=ks, v_scale=vs)
    model = [[([], [], []) for _ in range(H)] for _ in range(B)]      # cached keys, values, weights of the oracle
    exact = [[], []]
    for step in range(200):
        kv = [torch.randn(B, H, d, generator=g).to(IO[io]) for _ in range(2)]
        for r, x, e in zip(ring, kv, exact):
            r[:, step % wcap] = x.cuda()
            e.append(_f64(x))
        ctx += 1
        tail += 1
        q = (2 * torch.randn(B, 1, H * G, d, generator=g)).to(IO[io]).cuda()
        out, before = torch.empty_like(q), w.clone()
        L.lla_kv8_attn(q=q, out=out, lens=lens, win_k=ring[0], win_v=ring[1], ctx=ctx, tail=tail, weights=w, **cache)
        n, t = int(lens[0]), int(tail[0])
        if step % 13 == 0 or step > 190:
            c = Cache.__new__(Cache)
            c.k8, c.block = k8, block
            c.values = {m: [np.stack([np.array(model[b][h][i]).reshape(-1, d) for h in range(H)]) for b in range(B)]
                        for i, m in enumerate("kv")}
            assert c.values["k"][0].shape[1] == n
            _check(c, q, out, ring, [step + 1] * B, [t] * B, w, before)
        for b in range(B):
            for h in range(H):
                model[b][h][2][:] = _f64(w[b, h, :n]).tolist()
        if t == 32:                     # the oldest 16 of the exact tokens become a block
            L.lla_kv8_write(k=ring[0], v=ring[1], n=block, src0=ctx - tail, row0=lens, ring=True, **cache)
            for b in range(B):
                for h in range(H):
                    for i in range(2):
                        old = np.stack(exact[i][step + 1 - t:step + 1 - t + block])[:, b, h].astype(np.float32)
                        cc, s = kv8.write(old, block, code)
                        model[b][h][i].extend(kv8.values(cc, s, block))
                    model[b][h][2].extend([0.0] * block)
            lens += block
            tail -= block
        if int(lens[0]) == cap:
            before = w.cpu()
            L.lla_kv8_evict(**cache, weights=w, lens=lens, keep=keep, first=1, last=1)
            assert lens.tolist() == [keep * block] * B
            for b in range(B):
                for h in range(H):
                    ids = kv8.choose(before[b, h].numpy(), cap, block, keep, 1, 1)
                    rows = [i * block + j for i in ids for j in range(block)]
                    for i in range(3):
                        model[b][h][i][:] = [model[b][h][i][r] for r in rows]
                    assert np.array_equal(_f64(w[b, h, :keep * block]), np.array(model[b][h][2]))
            assert not w[:, :, keep * block:].any()


@pytest.mark.parametrize("win", ["f32", "bf16"])
@pytest.mark.parametrize("G,nq", [(1, 1), (8, 1), (2, 12), (32, 1)])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_f32_over_mostly_exact_tokens_keeps_its_precision(d, G, nq, win):
    """The error of the whole output in norm, where the sums' own roundings show and not single elements.  Logits of
    standard deviation 2: those that matter are about 4.5.  Added to nearest in D / 16 <= 16 steps a logit is off by
    sqrt(16) 2^-24 / sqrt(3) 2.6 = 3.6e-7, by 2^-24 times the spread of 2 for the truncated sums of 16, by 2^-25 4.5 for
    the rounding of the difference and 2^-22 / 3 for the exponential; the values' sum is off by less than the logits'.
    Added up as squares that is 5e-7; twice that is allowed."""
    B, H, W, T = 2, 3, 256, 250
    c = Cache(11, B, H, d, 32, 32, "i8", [20, 3])
    g = torch.Generator().manual_seed(d + G + nq)
    q = (2 * torch.randn(B, nq, H * G, d, generator=g)).cuda()
    ring = [torch.randn(B, W, H, d, generator=g).to(IO[win]).cuda() for _ in range(2)]
    ctx = [1000, 77777]
    out = _run_attn(c, q, ring, ctx, [T, T - 3])
    err = norm = 0.0
    for b, t in enumerate((T, T - 3)):
        wk, wv = (kv8.ring_rows(_f64(x[b]), ctx[b], t).reshape(t, H, d) for x in ring)
        ref, _ = kv8.attn(_f64(q[b]).reshape(nq, H, G, d), c.values["k"][b], c.values["v"][b], wk, wv)
        got = _f64(out[b]).reshape(ref.shape)
        err += np.sum((got - ref) ** 2)
        norm += np.sum(ref ** 2)
    assert math.sqrt(err / norm) <= 1e-6


@pytest.mark.parametrize("many_heads", [False, True])
def test_calls_on_two_streams_do_not_share_scratch(many_heads):
    """Each stream's call takes its own scratch although neither waits for the other: reads with weights (partial results
    and scores) and evictions of many heads (the list of blocks that stay)."""
    B, H, d, block, cap = 4, 40, 64, 32, 1024
    side, rounds = torch.cuda.Stream(), 20
    sets = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        k8, v8 = (torch.randint(-127, 128, (B, H, cap, d), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
        ks, vs = (torch.rand(B, H, cap // block, generator=g, device="cuda") * 0.02 for _ in range(2))
        q = torch.randn(B, 3, H, d, generator=g, device="cuda").to(torch.bfloat16)
        w = torch.rand(B, H, cap, generator=g, device="cuda")
        sets.append((dict(k8=k8, v8=v8, k_scale=ks, v_scale=vs), q, w))

    def buffers():
        if not many_heads:
            return [(torch.zeros_like(q), w.clone()) for _, q, w in sets]
        return [dict({n: torch.zeros_like(t[:, :, :t.shape[2] // 4]) for n, t in c.items()},
                     weights=torch.zeros(B, H, cap // 4, device="cuda"), lens=torch.zeros(B, dtype=torch.int32, device="cuda"))
                for c, _, _ in sets]

    def call(i, to, stream):
        c, q, w = sets[i]
        if many_heads:
            L.lla_kv8_evict(**c, weights=w, lens=lens, keep=8, first=1, last=1, to=to, stream=stream)
        else:
            L.lla_kv8_attn(q=q, out=to[0], lens=lens, weights=to[1], stream=stream, **c)

    lens = _i32([cap, cap - 5, 700, 900])
    if many_heads:
        assert L.lla_kv8_evict_workspace_bytes(**sets[0][0], weights=sets[0][2], lens=lens, keep=8) > 0
    want = buffers()
    for i in range(2):
        call(i, want[i], None)
        torch.cuda.synchronize()
    got = [buffers() for _ in range(rounds)]
    torch.cuda.synchronize()
    for r in range(rounds):
        call(0, got[r][0], None)
        call(1, got[r][1], side)
    torch.cuda.synchronize()
    for r in range(rounds):
        for i in range(2):
            a, b = got[r][i], want[i]
            for x, y in zip(a.values(), b.values()) if many_heads else zip(a, b):
                assert torch.equal(x, y)


def _one_hot(c, q, out, sc, win=None, ctx=None, tail=None):
    """Rows whose largest logit lies so far above the others, past what fp32 sums may be off by, that one token has all
    the weight: those outputs.  How many there are."""
    B, nq, HG, d = q.shape
    H = c.k8.shape[1]
    G, found = HG // H, 0
    q64, o64 = _f64(q).reshape(B, nq, H, G, d), _f64(out).reshape(B, nq, H, G, d)
    half = q.dtype == torch.bfloat16
    for b, p, h, g in np.ndindex(B, nq, H, G):
        k, v = c.values["k"][b][h], c.values["v"][b][h]
        if win:
            see = max(0, tail[b] - (nq - 1 - p))
            k, v = (np.concatenate([x, kv8.ring_rows(_f64(r[b]), ctx[b], tail[b])[:see, h]]) for x, r in zip((k, v), win))
        s = sc * (k @ q64[b, p, h, g])
        off = sc * (np.abs(k) @ np.abs(q64[b, p, h, g])).max() * (2.0 ** -21 + (d + 4) * 2.0 ** -23)
        top, second = np.sort(s)[::-1][:2]
        if top - second > 2 * off + 60 and top < 1e38:
            found += 1
            # probabilities in f16 under the block's scale, the output's own rounding
            tol = (2.0 ** -10 + 2.0 ** -8 if half else 2.0 ** -20) * np.abs(v[s.argmax()]).max()
            assert np.all(np.abs(o64[b, p, h, g] - v[s.argmax()]) <= tol)
    return found


HUGE = [2.0 ** e for e in (12, 24, 27, 30, 40, 60, 90, 110)]


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("G", [40, 100])
def test_many_rows_of_huge_logits_end_and_give_their_token(G, far):
    """Logits past 2^29, where fp32 neighbours lie further apart than the references' slack."""
    c = Cache(21, 2, 1, 64, 32, 320, "i8", [300, 140])
    if far:
        f = torch.tensor([2.0 ** e for e in (0, 20, -30, 5, 9, -12, 0, 3, -2, 1)], device="cuda")
        c.v_scale *= f
        c.values["v"] = [v * f.double().cpu().numpy()[np.arange(v.shape[1]) // 32][None, :, None] for v in c.values["v"]]
    g = torch.Generator().manual_seed(2)
    for factor in HUGE:
        q = (factor * torch.randn(2, 1, G, 64, generator=g)).to(torch.bfloat16).cuda()
        out = _run_attn(c, q)
        assert torch.isfinite(out).all()
        assert _one_hot(c, q, out, 1 / 8) >= G
        w = torch.zeros(2, 1, 320, device="cuda")
        _one_hot(c, q, _run_attn(c, q, weights=w), 1 / 8)
        assert abs(w.sum().item() - 2 * G) <= 2 * G * 2.0 ** -12


@pytest.mark.parametrize("G", [5, 40, 100])
def test_a_row_does_not_depend_on_the_other_rows_queries(G):
    """A padded row's query may hold anything: infinities, NaN, the type's largest value, values 2^60 times the others'."""
    c = Cache(7, 1, 2, 96, 32, 320, "e4m3", [300])
    q = torch.randn(1, 2, 2 * G, 96, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    q[0, :, 1::2] *= 2.0 ** -12
    clean = _run_attn(c, q)
    _check(c, q, clean)
    for bad in (math.nan, math.inf, -math.inf, torch.finfo(torch.bfloat16).max, 2.0 ** 60):
        odd = q.clone()
        odd[0, 1, 3] = bad
        odd[0, 0, G + 2, 17] = bad
        out = _run_attn(c, odd)
        same = torch.ones(2, 2 * G, dtype=torch.bool)
        same[1, 3] = same[0, G + 2] = False
        assert torch.equal(out[0][same], clean[0][same])
        if not math.isfinite(bad):
            assert not torch.isfinite(out[0][~same]).all(-1).any()


@pytest.mark.parametrize("ratio", [0.9, 5, 60, 900, 1e6])
@pytest.mark.parametrize("N", [700, 16384, 65536])
@pytest.mark.parametrize("G", [32, 40, 100])
def test_a_flat_rest_beside_a_peak_and_an_unattended_block(G, N, ratio):
    """One token 14.4 bits above the rest, which together outweigh it, and a block whose values are `ratio` times the
    others' and whose weight is nothing.  Probabilities are f16: 2^-11 each; those that f16 holds as subnormals, 2^-25
    under a largest of 2^2 or more in one sum."""
    d, block = 64, 64
    g = torch.Generator().manual_seed(N)
    k = torch.zeros(N, d, dtype=torch.int8)
    k[0, 0] = 80
    k[64:128, :2] = -127
    v = torch.randint(-67, 128, (N, d), generator=g, dtype=torch.int8)
    vs = torch.full((N // block + 1,), 0.01)
    vs[1] *= ratio
    q = torch.zeros(G, d)
    q[:, :2] = 1 + torch.randint(-8, 9, (G, 2), generator=g) / 128
    q = q.to(torch.bfloat16)
    cap = (N // block + 1) * block
    k8, v8 = (torch.nn.functional.pad(x, (0, 0, 0, cap - N))[None, None].cuda() for x in (k, v))
    out = torch.zeros(1, 1, G, d, dtype=torch.bfloat16, device="cuda")
    L.lla_kv8_attn(q=q[None, None].cuda(), out=out, lens=N, k8=k8, v8=v8, k_scale=torch.ones(1, 1, len(vs), device="cuda"),
                   v_scale=vs[None, None].cuda())
    val = v.double() * vs.double()[torch.arange(N) // block, None]
    a = torch.softmax(q.double() @ k.double().T / math.sqrt(d), -1)
    ref = a @ val
    bound = a @ val.abs() * 2.0 ** -10 + a[:, :1] * 1.27 * N * 2.0 ** -27 + ref.abs() * 2.0 ** -8
    assert ((out[0, 0].double().cpu() - ref).abs() <= bound).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("wdt", [None, "bf16", "f32"])
@pytest.mark.parametrize("G", [1, 5, 20])
def test_huge_logits_give_their_token(G, wdt, io):
    """As above in the kernel for few rows and among exact tokens; value scales from 2^-30 to 2^20."""
    c = Cache(22, 2, 2, 64, 32, 320, "e4m3", [300, 20])
    f = torch.tensor([2.0 ** e for e in (6, 20, -30, 5, 9, -12, 0, 3, -2, 1)], device="cuda")
    c.v_scale *= f
    c.values["v"] = [v * f.double().cpu().numpy()[np.arange(v.shape[1]) // 32][None, :, None] for v in c.values["v"]]
    g = torch.Generator().manual_seed(2)
    win = [_randn(g, 2, 128, 2, 64).to(IO[wdt]).cuda() for _ in range(2)] if wdt else None
    ctx, tail = [500, 77], [128, 70]
    for factor in HUGE:
        q = (factor * torch.randn(2, 3, 2 * G, 64, generator=g)).to(IO[io]).cuda()
        out = _run_attn(c, q, win, ctx, tail)
        assert torch.isfinite(out).all()
        assert _one_hot(c, q, out, 1 / 8, win, ctx, tail) >= 6 * G
        w = torch.zeros(2, 2, 320, device="cuda")
        _one_hot(c, q, _run_attn(c, q, win, ctx, tail, weights=w), 1 / 8, win, ctx, tail)
        assert torch.isfinite(w).all() and w.min() >= 0


@pytest.mark.parametrize("G", [2, 40])
def test_a_tail_longer_than_the_context_is_the_context(G):
    """A ring that is not full yet, read with tail = its size: slots that no position has reached hold NaN."""
    c = Cache(5, 3, 2, 64, 32, 96, "i8", [70, 0, 33])
    g = torch.Generator().manual_seed(1)
    ctx = [5, 0, 16]
    win = [torch.randn(3, 16, 2, 64, generator=g) for _ in range(2)]
    for b in range(3):
        for x in win:
            x[b, ctx[b]:] = math.nan
    win = [x.to(torch.bfloat16).cuda() for x in win]
    q = torch.randn(3, 3, 2 * G, 64, generator=g).to(torch.bfloat16).cuda()
    _check(c, q, _run_attn(c, q, win, ctx, [16, 16, 16]), win, ctx, ctx)
    _check(c, q, _run_attn(c, q, win, [-4, -1, 2], [1, 0, 9]), win, [0, 0, 2], [0, 0, 2])
    out = torch.zeros_like(q)
    L.lla_kv8_attn(q=q, out=out, lens=_i32(c.lens), win_k=win[0], win_v=win[1], ctx=2, tail=16, **c.args())
    again = _run_attn(c, q, win, [2, 2, 2], [2, 2, 2])
    assert torch.equal(out[::2], again[::2])


@pytest.mark.parametrize("H,keep", [(1, 8192), (1, 8191), (2, 6000), (149, 5), (149, 8000)])
def test_eviction_of_the_most_blocks(H, keep):
    """8192 blocks: keys and the list of kept blocks fill the most shared memory, with few heads and with many."""
    B, d, block, cap = 1, 16, 16, 8192 * 16
    g = torch.Generator(device="cuda").manual_seed(keep)
    n = cap - 5
    k8, v8 = (torch.randint(-127, 128, (B, H, cap, d), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand(B, H, cap // block, generator=g, device="cuda") for _ in range(2))
    w = torch.randint(0, 50, (B, H, cap), generator=g, device="cuda").float()     # sums are exact, and many are equal
    lens, kept = _i32([n]), torch.empty(B, H, keep, dtype=torch.int32, device="cuda")
    was = [t.clone() for t in (k8, v8, ks, vs, w)]
    L.lla_kv8_evict(k8=k8, v8=v8, k_scale=ks, v_scale=vs, weights=w, lens=lens, keep=keep, first=2, last=2, kept=kept)
    new = n - (8192 - keep) * block
    assert lens.tolist() == [new]
    mass = was[4].view(H, -1, block).sum(-1)
    mass[:, :2] = mass[:, -2:] = math.inf
    ids = mass.sort(dim=-1, descending=True, stable=True).indices[:, :keep].sort(-1).values
    assert torch.equal(kept[0].long(), ids)
    rows = (ids[..., None] * block + torch.arange(block, device="cuda")).flatten(1)[:, :new]
    for x, y in ((k8, was[0]), (v8, was[1])):
        assert torch.equal(x[0, :, :new], y[0].gather(1, rows[..., None].expand(-1, -1, d)))
    for x, y in ((ks, was[2]), (vs, was[3])):
        assert torch.equal(x[0, :, :keep], y[0].gather(1, ids))
    assert torch.equal(w[0, :, :new], was[4][0].gather(1, rows)) and not w[0, :, new:n].any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 5, 20, 40])
def test_weights_of_huge_logits_sum_to_the_rows(G, io):
    """A weight is formed from a kept score and the joined statistics, which must stand in the same units."""
    c = Cache(22, 2, 2, 64, 32, 320, "i8", [300, 20])
    g = torch.Generator().manual_seed(2)
    for factor in HUGE:
        q = (factor * torch.randn(2, 2, 2 * G, 64, generator=g)).to(IO[io]).cuda()
        w = torch.zeros(2, 2, 320, device="cuda")
        _run_attn(c, q, weights=w)
        # past 2^24 a logit's rounding is worth a bit and more: then only rows of one token say what a weight is
        off = factor * 40 * 2.0 ** -22 if factor < 2.0 ** 14 else 2.0 ** -16
        top, got = _tops(c, q), _f64(w)
        for b, h in np.ndindex(2, 2):
            sure = top[b][h] >= 0
            if sure.all():
                want = np.bincount(top[b][h], minlength=320)
                assert np.all(np.abs(got[b, h] - want) <= off * np.maximum(want, 1) + 2.0 ** -20)
        assert factor < 2.0 ** 14 or (top[1][0] >= 0).all()


def _tops(c, q):
    """[b][h]: for each row the token that has all its weight, -1 where none has beyond what fp32 sums may be off by."""
    B, nq, HG, d = q.shape
    H = c.k8.shape[1]
    q64 = _f64(q).reshape(B, nq, H, HG // H, d)
    out = []
    for b in range(B):
        per = []
        for h in range(H):
            k, r = c.values["k"][b][h], q64[b, :, h].reshape(-1, d)
            s = r @ k.T / math.sqrt(d)
            off = (np.abs(r) @ np.abs(k).T).max(1) / math.sqrt(d) * (2.0 ** -21 + (d + 4) * 2.0 ** -23)
            two = np.sort(s, 1)[:, -2:]
            per.append(np.where(two[:, 1] - two[:, 0] > 2 * off + 60, s.argmax(1), -1))
        out.append(per)
    return out


@pytest.mark.parametrize("bits", [22, 24, 25, 26, 28])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_flat_rest_far_below_a_peak(io, bits):
    """600 heads, so that one CTA sums a whole head and each warp a quarter: a peak and 65536 tokens `bits` below it, of
    values that the peak does not have.  One f16 term may lose 2^-25 under a largest of 2^2 of each, two a 2^-37."""
    H, N, d, block = 600, 65536, 64, 256
    g = torch.Generator().manual_seed(bits)
    k = torch.zeros(N, d, dtype=torch.int8)
    k[100, 0] = 100
    v = torch.randint(0, 128, (N, d), generator=g, dtype=torch.int8)
    v[:, 32:] = 100
    v[100, :32] = 0
    q = torch.zeros(1, 1, H, d, device="cuda")
    q[..., 0] = bits * math.log(2) * 8 / 100
    q = q.to(IO[io])
    out = torch.zeros_like(q)
    k8, v8 = (x[None, None].cuda().expand(1, H, N, d) for x in (k, v))      # all heads read the same rows
    ks, s = (torch.full((1, 1, N // block), x, device="cuda").expand(1, H, -1) for x in (1.0, 0.01))
    L.lla_kv8_attn(q=q, out=out, lens=N, k8=k8, v8=v8, k_scale=ks, v_scale=s)
    a = torch.softmax(float(q[0, 0, 0, 0]) * k[:, 0].double() / 8, 0)
    ref = a @ (v.double() * float(s[0, 0, 0]))
    # the weights: a logit of up to 28 bits, its product, sum and difference rounded, and sums of 65536 / 4 / 32 terms
    rel = 28 * 2.0 ** -22 + 2.0 ** -20 + 2048 * 2.0 ** -24 / 8
    lost = a.max().item() * 1.27 * N / 4 * (2.0 ** -27 if io == "bf16" else 2.0 ** -39)
    tol = ref * (rel + (2.0 ** -10 + 2.0 ** -8 if io == "bf16" else 0)) + lost
    assert ((out[0, 0].double().cpu() - ref).abs() <= tol).all()


def test_calls_on_forked_streams_of_one_capture():
    """Scratch of the call on the forked stream comes from the capture's memory and is not the other call's."""
    case = (3, 2, 2, 5, 64, 32, [900, 40, 640], "i8", "bf16", 16, [5, 9, 16], "bf16")
    sets = [_inputs(case, seed) for seed in (0, 50)]
    outs, before = [torch.zeros_like(s[1]) for s in sets], [s[5].clone() for s in sets]
    side = torch.cuda.Stream()
    args = [dict(q=q, out=o, lens=_i32(c.lens), win_k=win[0], win_v=win[1], ctx=_i32(ctx), tail=_i32(tails), weights=w,
                 **c.args()) for (c, q, win, ctx, tails, w), o in zip(sets, outs)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        L.lla_kv8_attn(**args[0])
        L.lla_kv8_attn(stream=side, **args[1])
        main.wait_stream(side)
    for _ in range(3):
        for (_, _, _, _, _, w), b in zip(sets, before):
            w.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for (c, q, win, ctx, tails, w), o, b in zip(sets, outs, before):
            _check(c, q, o, win, ctx, tails, w, b)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 40])
def test_values_near_the_largest_fp32_number(G, io):
    """An fp32 ring's value that bf16 terms cannot hold: kept out of the queries that do not see it, and met as it is by
    those that do."""
    c = Cache(3, 1, 2, 64, 32, 96, "i8", [70])
    g = torch.Generator().manual_seed(1)
    q = torch.randn(1, 3, 2 * G, 64, generator=g).to(IO[io]).cuda()
    win = [torch.randn(1, 8, 2, 64, generator=g).cuda() for _ in range(2)]
    clean = _run_attn(c, q, win, [90], [6])
    for bad in (torch.finfo(torch.float32).max, torch.finfo(torch.float32).min, 3.3961775e38):
        dirty = [win[0], win[1].clone()]
        dirty[1][0, 89 % 8, 1, 5] = bad                   # the last position, head 1
        out = _run_attn(c, q, dirty, [90], [6])
        # a tile of exact tokens is summed another way then
        assert (out[:, :2] - clean[:, :2]).abs().max() <= (2.0 ** -7 if io == "bf16" else 2.0 ** -19) * clean.abs().max()
        assert torch.equal(out[:, 2, :G], clean[:, 2, :G])
        kk, vv = (np.concatenate([x, kv8.ring_rows(_f64(r[0]), 90, 6)[:, 1]])
                  for x, r in zip((c.values["k"][0][1], c.values["v"][0][1]), dirty))
        for i in range(G):
            ref, a = kv8.attend(_f64(q[0, 2, G + i]), kk, vv)
            got = _f64(out[0, 2, G + i])
            assert abs(got[5] - ref[5]) <= (2.0 ** -7 if io == "bf16" else 2.0 ** -17) * abs(ref[5])
            assert np.all(np.abs(np.delete(got - ref, 5)) <= (2.0 ** -7 if io == "bf16" else 2.0 ** -17) * np.abs(vv[:, 6:]).max())
