"""Log probabilities of rows in sequences and at any element of a tensor: the bits of the same call on copies."""
import pytest
import torch

from test_gpu_token_logprobs import BF, F32, I32, random_logits

pytestmark = pytest.mark.gpu


def e(*shape, dtype=F32):
    """A tensor that starts one element past its memory's start."""
    n = 1
    for s in shape:
        n *= s
    return torch.full((n + 8,), -77, dtype=dtype, device="cuda")[1:n + 1].view(shape)


def forward(lib, x, t, top, make):
    lead = x.shape[:-1]
    rows = lead.numel()
    o = dict(logprob=make(*lead), entropy=make(*lead), stats=make(*lead, 2))
    if top:
        o |= dict(top_ids=make(*lead, top, dtype=I32), top_logprobs=make(*lead, top))
    need = lib.token_logprobs_workspace(rows, x.shape[-1], top)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    lib.token_logprobs(x, t, workspace=ws, scale=0.75, **o)
    return o


def backward(lib, x, t, o, d):
    lead = x.shape[:-1]
    w = torch.linspace(-1, 1, lead.numel(), device="cuda").view(lead)
    lib.token_logprobs_backward(x, t, o["stats"], dlogprob=w, entropy=o["entropy"], dentropy=w * 0.3, dlogits=d, scale=0.75)


def check(lib, x, t, d, top=5):
    """x, t and d are slices."""
    c = lambda v: v.contiguous().clone()
    plain = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")
    want, got = forward(lib, c(x), c(t), top, plain), forward(lib, x, t, top, e)
    assert all(torch.equal(got[k], want[k]) for k in want)
    wd = torch.empty_like(c(x))
    backward(lib, c(x), c(t), want, wd)
    backward(lib, x, t, got, d)
    assert torch.equal(d, wd) and bool((wd != 0).any())
    # in place, what lies between left as it was
    backward(lib, x, t, got, x)
    assert torch.equal(x, wd)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("seqs,length,vocab", [(3, 5, 1000), (3, 5, 1001), (4, 200, 2051), (300, 3, 33), (2, 9, 70001),
                                               (1, 9, 501), (7, 2, 64), (2, 600, 4097)])
def test_next_tokens(gpu_lib, seqs, length, vocab, dtype):
    """Each sequence's rows but the last, with its tokens but the first."""
    x = torch.from_numpy(random_logits(1, seqs * length, vocab)).to(dtype).cuda().view(seqs, length, vocab)
    ids = torch.randint(0, vocab, (seqs, length), device="cuda")
    ids[0, -1] = -100
    last = x[:, -1].clone()
    d = torch.full((seqs, length + 1, vocab + 3), 7.0, dtype=dtype, device="cuda")
    check(gpu_lib, x[:, :-1], ids[:, 1:], d[:, 1:-1, 2:-1])
    assert torch.equal(x[:, -1], last)
    edge = torch.ones_like(d, dtype=torch.bool)
    edge[:, 1:-1, 2:-1] = False
    assert bool((d[edge] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,vocab", [(9, 1001), (6, 40003), (700, 77)])
def test_rows_from_the_second_on(gpu_lib, rows, vocab, dtype):
    """One sequence: logits and gradients that start off 16 bytes, targets off 16, outputs off 16."""
    x = torch.from_numpy(random_logits(2, rows + 1, vocab)).to(dtype).cuda()
    ids = torch.randint(0, vocab, (rows + 1,), device="cuda")
    d = torch.full((rows + 2, vocab), 7.0, dtype=dtype, device="cuda")
    first = x[0].clone()
    check(gpu_lib, x[1:], ids[1:], d[1:-1])
    assert torch.equal(x[0], first) and bool((d[0] == 7.0).all()) and bool((d[-1] == 7.0).all())


def test_captured(gpu_lib):
    """Slices in a captured graph, replayed with other contents."""
    x = torch.randn(4, 33, 777, device="cuda")
    ids, d = torch.randint(0, 777, (4, 33), device="cuda"), torch.zeros(4, 33, 777, device="cuda")
    graph = torch.cuda.CUDAGraph()
    o = forward(gpu_lib, x[:, :-1], ids[:, 1:], 3, e)
    w = torch.linspace(-1, 1, 128, device="cuda").view(4, 32)
    step = lambda o, d: (gpu_lib.token_logprobs(x[:, :-1], ids[:, 1:], scale=0.75, **o),
                         gpu_lib.token_logprobs_backward(x[:, :-1], ids[:, 1:], o["stats"], dlogprob=w, dlogits=d, scale=0.75))
    with torch.cuda.graph(graph):
        step(o, d[:, :-1])
    for i in range(3):
        x.mul_(0.8)
        ids.copy_(ids.flip(1))
        want = {k: torch.empty_like(v) for k, v in o.items()}
        dw = torch.empty(4, 32, 777, device="cuda")
        step(want, dw)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], want[k]) for k in o) and torch.equal(d[:, :-1], dw) and bool((d[:, -1] == 0).all()), i


def test_sequences_past_32_bits(gpu_lib):
    """Sequences whose rows lie past 2^32 bytes have the bits of a small call on them."""
    seqs, length, vocab = 130, 257, 65537
    x = torch.empty(seqs, length, vocab, dtype=BF, device="cuda")
    x[-1] = torch.randn(length, vocab, device="cuda").to(BF)
    x[:-1] = x[-1]
    ids = torch.randint(0, vocab, (seqs, length), device="cuda")
    ids[:] = ids[-1]
    lp, st = torch.empty(seqs, length - 1, device="cuda"), torch.empty(seqs, length - 1, 2, device="cuda")
    gpu_lib.token_logprobs(x[:, :-1], ids[:, 1:], logprob=lp, stats=st)
    assert torch.equal(lp, lp[-1:].expand_as(lp))
    keep = x[-1].clone()
    gpu_lib.token_logprobs_backward(x[:, :-1], ids[:, 1:], st, dlogprob=torch.ones_like(lp), dlogits=x[:, :-1])
    small = torch.empty_like(keep[:-1])
    gpu_lib.token_logprobs_backward(keep[:-1], ids[-1, 1:], st[-1], dlogprob=torch.ones(length - 1, device="cuda"), dlogits=small)
    assert torch.equal(x[-1, :-1], small) and torch.equal(x[3, :-1], small) and torch.equal(x[-1, -1], keep[-1])
