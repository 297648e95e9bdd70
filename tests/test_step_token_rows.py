"""Log probabilities of rows in sequences, starting anywhere in a tensor: refusals of the C calls, and what the binding
makes of slices.  Without a GPU; the pointers are fake and never dereferenced."""
import pytest
import torch

if torch.cuda.is_available():
    pytest.skip("host-only validation tests (fake device pointers)", allow_module_level=True)

from bit_gradient_compression_amd import loco  # noqa: E402

OK, INV, ALIGN, UNSUP, HIP = (loco.LOCO_OK, loco.LOCO_ERR_INVALID, loco.LOCO_ERR_ALIGN, loco.LOCO_ERR_UNSUPPORTED,
                              loco.LOCO_ERR_HIP)
F32, BF16 = loco.LOCO_F32, loco.LOCO_BF16
P = [0x100000000 * (i + 1) for i in range(16)]  # fake, aligned, 4 GiB apart


@pytest.fixture(scope="module")
def lib():
    return loco.load()


def logp(lib, **kw):
    a = dict(x=P[0], dtype=BF16, seqs=3, rows=4, vocab=100, ld=100, sld=500, t=P[1], tld=5, scale=1.0, lp=P[2], h=P[3],
             st=P[4], top=3, ids=P[5], tl=P[6], ws=P[7], nws=1 << 30)
    a.update(kw)
    return lib.loco_token_logprobs_ex(*(a[k] for k in ("x", "dtype", "seqs", "rows", "vocab", "ld", "sld", "t", "tld", "scale",
                                                       "lp", "h", "st", "top", "ids", "tl", "ws", "nws")), None)


def lback(lib, **kw):
    a = dict(x=P[0], dtype=F32, seqs=3, rows=4, vocab=100, ld=100, sld=500, t=P[1], tld=5, scale=1.0, st=P[2], h=P[3],
             dl=P[4], dh=P[5], dx=P[6], dld=104, dsld=520)
    a.update(kw)
    return lib.loco_token_logprobs_backward_ex(*(a[k] for k in ("x", "dtype", "seqs", "rows", "vocab", "ld", "sld", "t", "tld",
                                                                "scale", "st", "h", "dl", "dh", "dx", "dld", "dsld")), None)


# A call that passes its checks fails at its launch, here where there is no device.
STEPS = [
    (dict(), HIP), (dict(seqs=-1), INV), (dict(rows=-1), INV), (dict(ld=99), INV), (dict(sld=399), INV), (dict(sld=400), HIP),
    (dict(sld=0), INV), (dict(sld=-500), INV), (dict(seqs=1, sld=0, tld=0), HIP), (dict(seqs=1, sld=-7, tld=-7), HIP),
    (dict(tld=3), INV), (dict(tld=4), HIP), (dict(tld=0), INV), (dict(tld=-5), INV), (dict(ld=120, sld=459), INV),
    (dict(ld=120, sld=460), HIP), (dict(sld=1 << 52), INV), (dict(tld=1 << 52), INV), (dict(seqs=1 << 41), INV),
    (dict(seqs=1 << 30, rows=8, sld=800, tld=8), UNSUP), (dict(seqs=0), OK), (dict(rows=0, x=None, t=None), OK),
    (dict(seqs=0, sld=0, tld=0), OK),
]


@pytest.mark.parametrize("kw,want", STEPS + [
    (dict(x=P[0] + 2), HIP), (dict(x=P[0] + 1), ALIGN), (dict(dtype=F32, x=P[0] + 4), HIP), (dict(dtype=F32, x=P[0] + 2), ALIGN),
    (dict(t=P[1] + 8), HIP), (dict(t=P[1] + 4), ALIGN), (dict(lp=P[2] + 4), HIP), (dict(lp=P[2] + 2), ALIGN),
    (dict(h=P[3] + 4), HIP), (dict(h=P[3] + 1), ALIGN), (dict(st=P[4] + 4), HIP), (dict(st=P[4] + 2), ALIGN),
    (dict(ids=P[5] + 4), HIP), (dict(ids=P[5] + 2), ALIGN), (dict(tl=P[6] + 4), HIP), (dict(tl=P[6] + 2), ALIGN),
    # the last element of the logits, and past it; a target of the last sequence
    (dict(lp=P[0] + 2 * (2 * 500 + 4 * 100) - 4), INV), (dict(lp=P[0] + 2 * (2 * 500 + 4 * 100)), HIP),
    (dict(lp=P[1] + 8 * (2 * 5 + 4) - 4), INV), (dict(lp=P[1] + 8 * (2 * 5 + 4)), HIP),
    (dict(h=P[2] + 4 * 11), INV), (dict(h=P[2] + 4 * 12), HIP), (dict(ids=P[4] + 4 * 23), INV), (dict(ids=P[4] + 4 * 24), HIP),
    (dict(top=33), UNSUP), (dict(top=-1), INV), (dict(vocab=(1 << 24) + 1, ld=1 << 25, sld=1 << 28), UNSUP),
    (dict(vocab=40000, ld=40000, sld=200000, nws=0), INV), (dict(vocab=40000, ld=40000, sld=200000, ws=P[7] + 8), ALIGN),
])
def test_token_logprobs_ex(lib, kw, want):
    assert logp(lib, **kw) == want


@pytest.mark.parametrize("kw,want", STEPS + [
    (dict(dld=99), INV), (dict(dsld=411), INV), (dict(dsld=412), HIP), (dict(dsld=1 << 52), INV), (dict(seqs=1, dsld=0), HIP),
    (dict(x=P[0] + 4), HIP), (dict(x=P[0] + 2), ALIGN), (dict(t=P[1] + 8), HIP), (dict(t=P[1] + 4), ALIGN),
    (dict(st=P[2] + 4), HIP), (dict(h=P[3] + 4), HIP), (dict(dl=P[4] + 4), HIP), (dict(dh=P[5] + 4), HIP),
    (dict(dx=P[6] + 4), HIP), (dict(dx=P[6] + 2), ALIGN), (dict(dtype=BF16, dx=P[6] + 2, x=P[0] + 6), HIP),
    (dict(dx=P[0]), INV), (dict(dx=P[0], dld=100, dsld=500), HIP), (dict(dx=P[0], dld=100, dsld=520), INV),
    (dict(seqs=1, dx=P[0], dld=100), HIP), (dict(dx=P[0] + 4 * 1400), HIP), (dict(dx=P[0] + 4 * 1399), INV),
    (dict(st=P[6] + 4 * (2 * 520 + 3 * 104 + 99)), INV), (dict(st=P[6] + 4 * (2 * 520 + 3 * 104 + 100)), HIP),
])
def test_token_logprobs_backward_ex(lib, kw, want):
    assert lback(lib, **kw) == want


class Calls:
    """In the library's place: keeps the layout of the last call."""

    def loco_token_logprobs_ex(self, x, dtype, seqs, rows, vocab, ld, sld, t, tld, *rest):
        self.got = (seqs, rows, vocab, ld, sld, tld)
        return 0

    def loco_token_logprobs_backward_ex(self, x, dtype, seqs, rows, vocab, ld, sld, t, tld, scale, st, h, dl, dh, dx, dld, dsld,
                                        stream):
        self.got = (seqs, rows, vocab, ld, sld, tld, dld, dsld)
        return 0


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(loco, "_device", lambda: -1)
    monkeypatch.setattr(loco, "_stream", lambda stream, dev: 0)
    monkeypatch.setattr(loco, "_lib", c)
    return c


def test_layouts_of_slices(calls):
    z = lambda *s: torch.zeros(*s)
    x, ids = z(5, 7, 11), torch.zeros(5, 7, dtype=torch.int64)
    lp = z(5, 6)

    def layout(logits, targets, n=None):
        loco.token_logprobs(logits, targets, logprob=z(n or logits.shape[:-1].numel()))
        return calls.got

    loco.token_logprobs(x[:, :-1], ids[:, 1:], logprob=lp)
    assert calls.got == (5, 6, 11, 11, 77, 7)
    assert layout(x, ids) == (1, 35, 11, 11, 0, 0)
    assert layout(x[:, :-1], ids[:, 1:].contiguous()) == (5, 6, 11, 11, 77, 6)
    assert layout(x[:, :-1].contiguous(), ids[:, 1:]) == (5, 6, 11, 11, 66, 7)
    assert layout(x[:, 1:, :9], ids[:, 1:]) == (5, 6, 9, 11, 77, 7)
    assert layout(x[..., :9], ids) == (1, 35, 9, 11, 385, 35)
    assert layout(x, torch.zeros(70, dtype=torch.int64)[::2]) == (35, 1, 11, 11, 11, 2)
    assert layout(x[:, ::2], ids[:, :4]) == (5, 4, 11, 22, 77, 7)
    assert layout(x[0, :-1], ids[0, 1:]) == (1, 6, 11, 11, 0, 0)
    assert layout(x[:, 3], ids[:, 3]) == (5, 1, 11, 77, 77, 7)
    assert layout(x[:, :1], ids[:, 1:2]) == (5, 1, 11, 77, 77, 7)
    assert layout(x[1:, 2:], ids[1:, 2:]) == (4, 5, 11, 11, 77, 7)
    assert layout(x[:1, :-1], ids[:1, 1:]) == (1, 6, 11, 11, 0, 0)
    assert layout(z(2, 5, 7, 11)[:, :, :-1], torch.zeros(2, 5, 7, dtype=torch.int64)[..., 1:]) == (10, 6, 11, 11, 77, 7)
    dx, st = torch.zeros(5, 7, 13), z(5, 6, 2)
    loco.token_logprobs_backward(x[:, :-1], ids[:, 1:], st, dlogprob=lp, dlogits=dx[:, :-1, :11])
    assert calls.got == (5, 6, 11, 11, 77, 7, 13, 91)
    loco.token_logprobs_backward(x[:, :-1], ids[:, 1:], st, dlogprob=lp, dlogits=x[:, :-1])
    assert calls.got == (5, 6, 11, 11, 77, 7, 11, 77)
    loco.token_logprobs_backward(x[:, :-1].contiguous(), ids[:, 1:].contiguous(), st, dlogprob=lp, dlogits=z(5, 6, 11))
    assert calls.got == (1, 30, 11, 11, 0, 0, 11, 0)
    loco.token_logprobs_backward(x[:, :-1].contiguous(), ids[:, 1:].contiguous(), st, dlogprob=lp, dlogits=dx[:, 1:, :11])
    assert calls.got == (5, 6, 11, 11, 66, 6, 13, 91)


def test_refused_slices(calls):
    z = lambda *s: torch.zeros(*s)
    x, ids = z(5, 7, 11), torch.zeros(5, 7, dtype=torch.int64)

    def refused(match, fn, *a, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)

    f, g = loco.token_logprobs, loco.token_logprobs_backward
    refused("apart", f, x.transpose(0, 1), ids.t().contiguous(), logprob=z(35))
    refused("apart", f, z(3, 5, 7, 11)[:, :-1, :-1], torch.zeros(72, dtype=torch.int64), logprob=z(72))
    refused("apart", f, z(7, 11).expand(5, 7, 11), ids, logprob=z(35))
    refused("apart", f, torch.as_strided(x, (5, 7, 11), (60, 11, 1)), ids, logprob=z(35))  # sequences that overlap
    refused("contiguous", f, x, ids[:, :1].expand(5, 7), logprob=z(35))
    refused("contiguous", f, x, torch.zeros(7, 5, dtype=torch.int64).t(), logprob=z(35))
    refused("contiguous", f, x, torch.as_strided(ids, (5, 7), (3, 1)), logprob=z(35))
    refused("contiguous", f, x[:, :-1], ids[:, 1:], logprob=z(5, 7)[:, 1:])
    # sequences of two rows and of four
    a, b = torch.as_strided(z(800), (2, 2, 2, 8), (200, 100, 8, 1)), torch.as_strided(z(800), (2, 2, 2, 8), (200, 16, 8, 1))
    refused("sequences of 2 and 4 rows", g, a, None, z(8, 2), dentropy=z(8), entropy=z(8), dlogits=b)
