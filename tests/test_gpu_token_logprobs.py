"""Log probabilities of tokens, entropy, alternatives and their gradient, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from layer_util import U, Guarded, assert_near, f64, guarded, round_bound
from oracle import step_oracle as O

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
INF = float("inf")

VOCABS = [1, 2, 7, 8, 9, 64, 65, 500, 513, 2047, 2048, 2049, 5003, 8191, 8192, 8195, 32000, 50001, 131071, 262147]


class Rows:
    """Logits between guards, in rows `pad` elements longer than the vocabulary."""

    def __init__(self, values, dtype, pad=0):
        values = torch.as_tensor(values, dtype=torch.float64)
        self.rows, self.vocab = values.shape
        self.g = Guarded((self.rows, self.vocab + pad), dtype, 7.0)
        self.x = self.g.t[:, :self.vocab]
        self.x.copy_(values.to(dtype))

    def check(self):
        self.g.check()
        assert bool((self.g.t[:, self.vocab:] == 7.0).all())


def random_logits(seed, rows, vocab, spread=3.0):
    r = np.random.default_rng(seed)
    return r.normal(size=(rows, vocab)) * spread * np.exp(0.4 * r.normal(size=(rows, 1)))


def random_targets(seed, rows, vocab):
    t = np.random.default_rng(seed + 1).integers(0, vocab, size=rows)
    if rows > 2:
        t[1] = -100
    return t


def additions(vocab):
    """Additions and changes of the maximum that a term passes through: batches of one lane (of 512
    values at least for the 64 lanes of a small vocabulary), the lanes and waves."""
    return 7 * (vocab / 2048 + 20) + 60


def forward_bounds(x, targets, scale, o):
    """Roundings: d = x - m, its product with the scale and log2 e, the exponential (3 |scale d| + 4
    units of e), a factor of the same kind at each change of the maximum, the additions; a
    logarithm within two units."""
    with np.errstate(all="ignore"):
        m, s = o["stats"][:, 0], o["stats"][:, 1]
        d = np.where(np.isfinite(x), x - m[:, None], 0.0)
        e = np.where(np.isfinite(x), np.exp(scale * d), 0.0)
        n = additions(x.shape[1])
        ad = scale * np.abs(d)
        rel = U * ((e * 3 * ad).sum(1) / s + n)
        dls = rel + 4 * U * np.abs(np.log(s)) + 2 * U
        dt = U * (e * np.abs(d) * (3 * ad + n)).sum(1)
        h = dls + scale * (dt / s + (e * np.abs(d)).sum(1) / s * (rel + 4 * U)) + 2 * U * np.abs(o["entropy"])
        own = np.abs(scale * (x[np.arange(len(x)), np.clip(targets, 0, x.shape[1] - 1)] - m))
        lp = dls + 3 * U * np.where(np.isfinite(own), own, 0.0) + 2 * U * np.abs(o["logprob"])
        k = o["top_logprobs"]
        tops = dls[:, None] + 4 * U * (np.abs(k) + np.abs(np.log(s))[:, None])
        clean = lambda b: np.where(np.isfinite(b), b, 0.0)
    return dict(stats=np.stack([np.zeros_like(s), clean(rel * s)], 1), entropy=clean(h), logprob=clean(lp),
                top_logprobs=clean(tops))


def run_forward(lib, x, targets, scale, top, entropy=True, stats=True, logprob=True):
    rows, vocab = x.shape
    t = torch.from_numpy(targets).cuda()
    g = dict(logprob=guarded((rows,), F32) if logprob else None, entropy=guarded((rows,), F32) if entropy else None,
             stats=guarded((rows, 2), F32) if stats else None, top_ids=guarded((rows, top), I32) if top else None,
             top_logprobs=guarded((rows, top), F32) if top else None)
    need = lib.token_logprobs_workspace(rows, vocab, top)
    ws = Guarded((need,), torch.uint8, 0xCC) if need else None
    lib.token_logprobs(x, t if logprob else None, scale=scale, workspace=ws.t if ws else None,
                       **{k: None if v is None else v.t for k, v in g.items()})
    torch.cuda.synchronize()
    for v in [*g.values(), ws]:
        if v is not None:
            v.check()
    return {k: v.t for k, v in g.items() if v is not None}


def check_forward(lib, logits, dtype, top=0, scale=1.0, pad=0, targets=None, seed=0, **parts):
    a = Rows(logits, dtype, pad)
    targets = random_targets(seed, a.rows, a.vocab) if targets is None else np.asarray(targets)
    got = run_forward(lib, a.x, targets, scale, top, **parts)
    a.check()
    x = f64(a.x)
    scale = float(np.float32(scale))
    want = O.token_logprobs(x, targets, scale, top)
    bound = forward_bounds(x, targets, scale, want)
    for k, v in got.items():
        if k == "top_ids":
            assert np.array_equal(v.cpu().numpy(), want[k]), k
        else:
            # past the midpoint between fp32's largest number and 2^128 the nearest fp32 number is infinite
            w = np.where(np.abs(want[k]) >= 2.0 ** 128 - 2.0 ** 103, np.copysign(INF, want[k]), want[k])
            assert_near(v, w, bound[k] + 2 * U * np.abs(np.nan_to_num(w, posinf=0, neginf=0)), k)
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", VOCABS)
def test_forward(gpu_lib, vocab, dtype):
    """Few rows and many, alternatives or none, an inverse temperature, padded rows."""
    for i, (rows, top, scale, pad) in enumerate(((1, 8, 1.0, 0), (5, 0, 0.5, 3), (3, 32, 1.25, 0), (600, 5, 1.0, 1))):
        if rows * vocab > 20_000_000:
            rows = 20
        check_forward(gpu_lib, random_logits(vocab + i, rows, vocab), dtype, top, scale, pad, seed=i)


@pytest.mark.parametrize("vocab", [6, 1000, 40000])
def test_forward_parts(gpu_lib, vocab):
    """Each output by itself has the bits that it has among the others."""
    for rows in (3, 520):
        a = Rows(random_logits(1, rows, vocab), BF)
        t = random_targets(2, rows, vocab)
        whole = run_forward(gpu_lib, a.x, t, 1.0, 4)
        for keep in ("logprob", "entropy", "stats", "top"):
            got = run_forward(gpu_lib, a.x, t, 1.0, 4 if keep == "top" else 0, **{k: k == keep for k in
                                                                                  ("logprob", "entropy", "stats")})
            assert got
            for k, v in got.items():
                assert torch.equal(v, whole[k]), k


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,vocab", [(12, 40), (12, 3000), (12, 70001), (600, 9001)])
def test_masks(gpu_lib, rows, vocab, dtype):
    """Tokens masked with minus infinity, with the type's lowest value, both; all of them; a given token
    that is masked; one token left; values near the largest."""
    lo = float(torch.finfo(dtype).min)
    x = random_logits(3, rows, vocab)
    t = random_targets(4, rows, vocab)
    keep = min(vocab - 1, 17)
    x[0, keep:] = -INF
    x[1, keep:] = lo
    x[2, :] = -INF
    x[3, :] = lo
    x[4, ::2] = -INF
    x[4, 1::4] = lo
    x[5, :] = -INF
    x[5, vocab - 1] = 2.5
    x[6, :] = -INF
    x[6, 0] = lo
    x[7, 1:] = lo
    x[7, 0] = -lo
    x[8, keep:] = -INF
    t[:9] = [0, keep, 1, 2, 1, vocab - 1, 0, 1, vocab - 1]
    for scale in (1.0, 0.5):
        for top in (0, 5, 32):
            check_forward(gpu_lib, x, dtype, top, scale, targets=t)


@pytest.mark.parametrize("rows,vocab", [(9, 33), (9, 5000), (9, 33001), (600, 3000)])
def test_rows_without_a_distribution(gpu_lib, rows, vocab):
    x = random_logits(5, rows, vocab)
    x[1, vocab // 2] = np.nan
    x[2, vocab - 1] = INF
    x[3, 0], x[3, 1] = INF, -INF
    x[4, :] = np.nan
    x[5, :-1] = -INF
    x[5, -1] = np.nan
    for dtype in (BF, F32):
        for top in (0, 3):
            check_forward(gpu_lib, x, dtype, top)


def test_targets_out_of_range(gpu_lib):
    x = random_logits(6, 7, 1000)
    t = np.array([-1, 1000, 999, -(1 << 40), 1 << 40, 0, (1 << 32) + 5])
    got = check_forward(gpu_lib, x, BF, targets=t)
    assert torch.isnan(got["logprob"]).tolist() == [False, True, False, False, True, False, True]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [2, 600])
@pytest.mark.parametrize("vocab", [5, 31, 300, 2049, 8300, 40000, 140001])
def test_alternatives_in_hard_orders(gpu_lib, vocab, rows, dtype):
    """Ties at the lower index: all equal, two values, plus and minus zero; rising and falling rows; all
    the large values in the chunks of one lane or one group of lanes, more of them than are ranked at once."""
    if rows * vocab > 20_000_000:
        rows = 130
    i = np.arange(vocab)
    shapes = [np.zeros(vocab), np.where(i % 3 == 1, 1.0, 0.5), np.where(i % 2, 0.0, -0.0), i * 1e-3, -i * 1e-3]
    for lanes in (64, 256, 1024):
        shapes.append(np.where(i // 8 % lanes == 3, 5.0 + i / vocab, -i / vocab))
        shapes.append(np.where(i // 8 % lanes < lanes // 16, 5.0 - i / vocab, 0.0))
    shapes.append(np.where(i >= vocab - 40, 1.0 + i / vocab, 0.0))
    x = np.stack([shapes[r % len(shapes)] for r in range(max(rows, len(shapes)))])
    for top in (1, 7, 32):
        check_forward(gpu_lib, x[:rows] if rows > 2 else x, dtype, top)


@pytest.mark.parametrize("scale", [1e-6, 1e-3, 100.0, 1e6])
def test_scales(gpu_lib, scale):
    x = random_logits(8, 6, 4099)
    x[1] *= 1e4
    x[2] = 3.0
    for dtype in (BF, F32):
        check_forward(gpu_lib, x, dtype, 5, scale)


# -- backward -----------------------------------------------------------------------------

def backward_bounds(x, targets, scale, o, dlp, dh):
    """Roundings of d, the exponential and the sum's reciprocal (3 |scale d| + 10 units of p, with the
    sum's own rounding to fp32), and of the factor beside p, whose terms may cancel."""
    with np.errstate(all="ignore"):
        m, s = o["stats"][:, :1], o["stats"][:, 1:]
        d = np.where(np.isfinite(x), x - m, 0.0)
        p = np.where(np.isfinite(x), np.exp(scale * d) / s, 0.0)
        ad = scale * np.abs(d)
        a = np.zeros((len(x), 1)) if dlp is None else np.where(targets < 0, 0.0, np.abs(dlp))[:, None]
        f, df = a, 3 * U * a
        if dh is not None:
            h, ent, ls = np.abs(dh)[:, None], np.abs(o["entropy"])[:, None], np.abs(np.log(s))
            f = f + h * (ad + ls + ent)
            df = df + U * h * (6 * ent + 8 * ls + 8 * ad + 8)
        b = scale * p * (U * (3 * ad + 12) * f + df)
        good = (targets >= 0) & (targets < x.shape[1])
        at = np.arange(len(x))[good], targets[good]
        b[at] += 4 * U * scale * a[good, 0]
        # an exponential below the smallest normal number may be 0
        b = b + 2.0 ** -126 * scale * f
    return np.where(np.isfinite(b), b, 0.0)


def run_backward(lib, x, targets, scale, o, dlp, dh, pad=0, in_place=False):
    c = lambda v: None if v is None else torch.from_numpy(np.asarray(v)).float().cuda()
    out = None if in_place else Rows(np.zeros(x.shape), x.dtype, pad)
    d = x if in_place else out.x
    if not in_place:
        d.fill_(float("nan"))
    lib.token_logprobs_backward(x, None if targets is None else torch.from_numpy(targets).cuda(), c(o["stats"]),
                                dlogprob=c(dlp), entropy=c(o["entropy"]) if dh is not None else None, dentropy=c(dh),
                                dlogits=d, scale=scale)
    torch.cuda.synchronize()
    if out is not None:
        out.check()
    return d


def check_backward(lib, logits, dtype, scale=1.0, pad=0, entropy=True, logprob=True, targets=None, seed=0):
    a = Rows(logits, dtype, pad)
    x = f64(a.x)
    r = np.random.default_rng(seed)
    targets = random_targets(seed, a.rows, a.vocab) if targets is None else np.asarray(targets)
    f32 = lambda v: v.astype(np.float32).astype(np.float64)
    dlp = f32(r.normal(size=a.rows) / a.rows) if logprob else None
    dh = f32(r.normal(size=a.rows) * 0.1 / a.rows) if entropy else None
    o = O.token_logprobs(x, targets, scale, 0)
    want = O.token_logprobs_backward(x, targets if logprob else np.full(a.rows, -1), scale, dlp, dh)
    bound = backward_bounds(x, targets, scale, o, dlp, dh)
    got = run_backward(lib, a.x, targets if logprob else None, scale, o, dlp, dh, pad)
    a.check()
    assert_near(got, want, bound + round_bound(want, dtype), "dlogits")
    here = run_backward(lib, a.x, targets if logprob else None, scale, o, dlp, dh, in_place=True)
    a.check()
    same = (here == got) | (torch.isnan(here) & torch.isnan(got))
    assert bool(same.all()), "in place"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", VOCABS)
def test_backward(gpu_lib, vocab, dtype):
    for i, (rows, scale, pad, parts) in enumerate(((1, 1.0, 0, dict()), (5, 0.5, 3, dict(entropy=False)),
                                                   (3, 1.25, 1, dict(logprob=False)), (600, 1.0, 0, dict()))):
        if rows * vocab > 20_000_000:
            rows = 20
        check_backward(gpu_lib, random_logits(vocab + i, rows, vocab), dtype, scale, pad, seed=i, **parts)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("entropy", [False, True])
def test_backward_of_masks_and_lost_rows(gpu_lib, dtype, entropy):
    lo = float(torch.finfo(dtype).min)
    vocab = 9000
    x = random_logits(9, 12, vocab)
    x[0, 17:] = -INF
    x[1, 17:] = lo
    x[2, :] = -INF
    x[3, :] = lo
    x[4, 5] = np.nan
    x[5, 5] = INF
    x[6, :] = -INF
    x[6, 44] = 1.0
    x[8, :] = np.nan
    t = np.array([3, 3, 3, 3, 3, 3, 44, vocab, -1, -7, 0, vocab - 1])
    check_backward(gpu_lib, x, dtype, entropy=entropy, targets=t)


def test_gradient_is_that_of_the_forward_pass(gpu_lib):
    """In fp32, the change of a loss of log probabilities and entropies between two nearby sets of logits
    is what the gradient says, within 1 % (the step's square and 2^-24 of the terms are far below)."""
    rows, vocab, scale = 9, 777, 0.8
    x = torch.from_numpy(random_logits(11, rows, vocab)).float().cuda()
    t = random_targets(12, rows, vocab)
    r = np.random.default_rng(13)
    dlp, dh = (torch.from_numpy(r.normal(size=rows)).float().cuda() for _ in range(2))
    got = run_forward(gpu_lib, x, t, scale, 0)
    g = torch.empty_like(x)
    gpu_lib.token_logprobs_backward(x, torch.from_numpy(t).cuda(), got["stats"], dlogprob=dlp, entropy=got["entropy"],
                                    dentropy=dh, dlogits=g, scale=scale)
    d = torch.from_numpy(r.normal(size=(rows, vocab)) * 0.02).float().cuda()

    def loss(y):
        o = run_forward(gpu_lib, y, t, scale, 0)
        return float((o["logprob"].double() * dlp + o["entropy"].double() * dh).sum())

    diff, terms = (loss(x + d) - loss(x - d)) / 2, g.double() * d
    assert abs(diff - float(terms.sum())) <= 0.01 * float(terms.abs().sum())


def test_shapes_and_strides(gpu_lib):
    """Leading dimensions, a slice of padded rows of them, one row, no rows, every second row."""
    big = torch.randn(3, 4, 1100, device="cuda")
    x = big[..., :1001]
    t = torch.randint(0, 1001, (3, 4), device="cuda")
    lp, st = torch.empty(3, 4, device="cuda"), torch.empty(3, 4, 2, device="cuda")
    ids, tops = torch.empty(3, 4, 6, dtype=I32, device="cuda"), torch.empty(3, 4, 6, device="cuda")
    gpu_lib.token_logprobs(x, t, logprob=lp, stats=st, top_ids=ids, top_logprobs=tops)
    flat = x.reshape(12, 1001).contiguous()
    lp2, ids2 = torch.empty(12, device="cuda"), torch.empty(12, 6, dtype=I32, device="cuda")
    gpu_lib.token_logprobs(flat, t.view(-1), logprob=lp2, top_ids=ids2, top_logprobs=torch.empty(12, 6, device="cuda"))
    assert torch.equal(lp.view(-1), lp2) and torch.equal(ids.view(12, 6), ids2)
    d = torch.zeros_like(big)
    gpu_lib.token_logprobs_backward(x, t, st, dlogprob=torch.ones_like(lp), dlogits=d[..., :1001])
    d2 = torch.empty_like(flat)
    gpu_lib.token_logprobs_backward(flat, t.view(-1), st.view(12, 2), dlogprob=torch.ones_like(lp2), dlogits=d2)
    assert torch.equal(d[..., :1001].reshape(12, 1001), d2) and bool((d[..., 1001:] == 0).all())
    half = flat[::2]
    lp3 = torch.empty(6, device="cuda")
    gpu_lib.token_logprobs(half, t.view(-1)[::2].contiguous(), logprob=lp3)
    assert torch.equal(lp3, lp2[::2])
    one = torch.empty(1, device="cuda")
    gpu_lib.token_logprobs(flat[4:5][:, :1001], t.view(-1)[4:5], logprob=one)
    assert torch.equal(one, lp2[4:5])
    e = torch.empty(0, device="cuda")
    gpu_lib.token_logprobs(flat[:0], t.view(-1)[:0], logprob=e)
    gpu_lib.token_logprobs_backward(flat[:0], t.view(-1)[:0], torch.empty(0, 2, device="cuda"), dlogprob=e, dlogits=d2[:0])
    with pytest.raises(ValueError, match="apart"):
        gpu_lib.token_logprobs(flat.t(), torch.zeros(1001, dtype=torch.int64, device="cuda"),
                               logprob=torch.empty(1001, device="cuda"))


def test_offsets_past_32_bits(gpu_lib):
    """Rows past 2^32 bytes have the results of a small call on them."""
    rows, vocab = 33_001, 131_071
    x = torch.empty(rows, vocab, dtype=BF, device="cuda")
    x[-3:] = torch.randn(3, vocab, device="cuda").to(BF)
    x[:-3] = x[-1]
    t = torch.zeros(rows, dtype=torch.int64, device="cuda")
    t[-3:] = torch.tensor([5, vocab - 1, 70000])
    lp, st = torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    ids, tops = torch.empty(rows, 4, dtype=I32, device="cuda"), torch.empty(rows, 4, device="cuda")
    gpu_lib.token_logprobs(x, t, logprob=lp, stats=st, top_ids=ids, top_logprobs=tops)
    want = O.token_logprobs(f64(x[-3:]), t[-3:].cpu().numpy(), 1.0, 4)
    b = forward_bounds(f64(x[-3:]), t[-3:].cpu().numpy(), 1.0, want)
    assert_near(lp[-3:], want["logprob"], b["logprob"] + 2 * U * np.abs(want["logprob"]), "far rows")
    assert np.array_equal(ids[-3:].cpu().numpy(), want["top_ids"])
    assert bool((ids[:-3] == ids[-1]).all())
    keep = x[-3:].clone()
    gpu_lib.token_logprobs_backward(x, t, st, dlogprob=torch.ones_like(lp), dlogits=x)
    small = torch.empty_like(keep)
    gpu_lib.token_logprobs_backward(keep, t[-3:].contiguous(), st[-3:].contiguous(), dlogprob=torch.ones(3, device="cuda"),
                                    dlogits=small)
    assert torch.equal(x[-3:], small)


def test_streams_and_graphs(gpu_lib):
    """Another stream; two captured graphs that share a workspace, replayed with the program's own work
    between; the same call gives the same bits."""
    for rows, vocab, top in ((3, 50001, 20), (700, 4000, 3)):
        x = torch.from_numpy(random_logits(20, rows, vocab)).to(BF).cuda()
        t = random_targets(21, rows, vocab)
        tt = torch.from_numpy(t).cuda()
        want = run_forward(gpu_lib, x, t, 1.0, top)
        need = gpu_lib.token_logprobs_workspace(rows, vocab, top)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        new = lambda: {k: torch.zeros_like(v) for k, v in want.items()}
        out, side = new(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        gpu_lib.token_logprobs(x, tt, workspace=ws, stream=side, **out)
        side.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)
        graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], [new(), new()]
        grads = [torch.zeros_like(x) for _ in range(2)]
        one = torch.ones(rows, device="cuda")
        for g, o, d in zip(graphs, outs, grads):
            with torch.cuda.graph(g):
                gpu_lib.token_logprobs(x, tt, workspace=ws, **o)
                gpu_lib.token_logprobs_backward(x, tt, o["stats"], dlogprob=one, entropy=o["entropy"], dentropy=one, dlogits=d)
        for i in range(3):
            x.mul_(0.75)
            want = run_forward(gpu_lib, x, t, 1.0, top)
            for g in graphs:
                g.replay()
            torch.cuda.synchronize()
            for o in outs:
                assert all(torch.equal(o[k], want[k]) for k in want), i
            assert torch.equal(*grads) and bool((grads[0] != 0).any())
