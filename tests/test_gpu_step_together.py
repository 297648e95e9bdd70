"""The step operators one after another as a training step uses them, with the layer operators between:
a block's output normed, gated and added to the stream, normed for the head and checkpointed; the
head's log probabilities; the gradients back through all of it; AdamW over every parameter."""
import numpy as np
import pytest
import torch

from layer_util import f64
from oracle import layer_oracle as L
from oracle import step_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T, H, V = 390, 256, 1003
HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8)
SCALE, ENTROPY = 0.6, 0.01


def e(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def ckpt(rows, cols):
    return e(rows, cols, dtype=torch.int8), e(rows, -(-cols // 64), dtype=torch.uint8)


class Step:
    """stream + scale gate norm(stream W^T) -> norm -> head -> log probabilities, and back."""

    SHAPES = {"w": (H, H), "post": (H,), "gate": (H,), "norm": (H,), "head": (V, H)}

    def __init__(self, lib, state_bits, seed=0):
        self.lib, self.bits = lib, state_bits
        g = torch.Generator("cuda").manual_seed(seed)
        randn = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(BF)
        self.x, self.targets = randn(T, H), torch.randint(0, V, (T,), generator=g, device="cuda")
        self.targets[::7] = -1
        self.p = {"w": randn(H, H, scale=H ** -0.5), "post": 1 + randn(H, scale=0.1), "gate": 0.5 + randn(H, scale=0.2),
                  "norm": 1 + randn(H, scale=0.1), "head": randn(V, H, scale=2 * H ** -0.5)}
        self.g = {k: e(*s) for k, s in self.SHAPES.items()}
        self.master = {k: v.float() for k, v in self.p.items()}
        zeros = lambda n, dtype: torch.zeros(n, dtype=dtype, device="cuda")
        self.states = {}
        for k, v in self.p.items():
            n = v.numel()
            nb = -(-n // 256)
            if state_bits == 32:
                self.states[k] = zeros(n, F32), zeros(n, F32)
            else:
                self.states[k] = ((zeros(n, torch.uint8).view(torch.float8_e4m3fn), zeros(nb, torch.uint8)),
                                  (zeros(n, torch.uint8), zeros(nb, torch.uint8)))
        self.tensors = lib.AdamwTensors([(self.master[k], self.g[k], *self.states[k], self.p[k],
                                          0.1 if k in ("w", "head") else 0.0) for k in self.p])
        self.xq, self.outq = ckpt(T, H), ckpt(T, H)
        self.y, self.h, self.out, self.logits = e(T, H), e(T, H), e(T, H), e(T, V)
        self.rp, self.r, self.lp, self.ent = (e(T, dtype=F32) for _ in range(4))
        self.stats = e(T, 2, dtype=F32)
        self.ids, self.tops = e(T, 4, dtype=torch.int32), e(T, 4, dtype=F32)
        self.dout, self.dy, self.dx = e(T, H), e(T, H), e(T, H)
        scored = int((self.targets >= 0).sum())
        self.dlp = torch.full((T,), -1.0 / scored, device="cuda")
        self.dent = torch.full((T,), -ENTROPY / scored, device="cuda")
        need = max(lib.linear_workspace(T, H, H), lib.linear_workspace(T, V, H), lib.linear_input_grad_workspace(T, V, H),
                   lib.linear_weight_grad_workspace(T, V, H), lib.linear_weight_grad_workspace(T, H, H),
                   lib.residual_norm_backward_workspace(T, H), lib.token_logprobs_workspace(T, V, 4), 16)
        self.ws = e(need, dtype=torch.uint8)

    def gradients(self):
        lib, p, g, ws = self.lib, self.p, self.g, self.ws
        lib.checkpoint_write(self.x, codes=self.xq[0], exps=self.xq[1])
        lib.linear(self.x, p["w"], out=self.y, workspace=ws)
        lib.residual_norm(self.y, self.x, h=self.h, out=self.out, rstd=self.r, weight=p["norm"], post_rstd=self.rp,
                          post_weight=p["post"], gate=p["gate"], scale=SCALE, checkpoint=self.outq)
        lib.linear(self.out, p["head"], out=self.logits, workspace=ws)
        lib.token_logprobs(self.logits, self.targets, logprob=self.lp, entropy=self.ent, stats=self.stats, top_ids=self.ids,
                           top_logprobs=self.tops, workspace=ws)
        # the gradient takes the logits' place
        lib.token_logprobs_backward(self.logits, self.targets, self.stats, dlogprob=self.dlp, entropy=self.ent,
                                    dentropy=self.dent, dlogits=self.logits)
        lib.linear_weight_grad(self.logits, self.outq, out=g["head"], workspace=ws)
        lib.linear_input_grad(self.logits, p["head"], out=self.dout, workspace=ws)
        lib.residual_norm_backward(self.dout, self.h, rstd=self.r, weight=p["norm"], y=self.y, post_rstd=self.rp,
                                   post_weight=p["post"], gate=p["gate"], scale=SCALE, dresidual=self.dx, dy=self.dy,
                                   dgate=g["gate"], dweight=g["norm"], dpost_weight=g["post"], workspace=ws)
        lib.linear_weight_grad(self.dy, self.xq, out=g["w"], workspace=ws)

    def step(self, t):
        self.gradients()
        self.lib.adamw(self.tensors, step=t, **HP)

    def results(self):
        out = [self.lp, self.ent, self.ids, self.tops, self.dx, *self.g.values(), *self.master.values(), *self.p.values()]
        return [t.clone() for t in out]


def test_gradients(gpu_lib):
    """Each gradient within 5 % in norm of the 64-bit formulas on unrounded intermediates: each tensor
    of the chain is rounded to bf16 (2^-9 of a value at random) and the checkpoints to 8 bits (about 1 %)."""
    s = Step(gpu_lib, 32)
    s.gradients()
    torch.cuda.synchronize()
    p, x, t = {k: f64(v) for k, v in s.p.items()}, f64(s.x), s.targets.cpu().numpy()
    y = L.linear(x, p["w"], None, "none", None)[0]
    out, h, r, rp = O.residual_norm(y, x, p["norm"], p["post"], p["gate"], SCALE, 1e-5, True)
    logits = out @ p["head"].T
    o = O.token_logprobs(logits, t, 1.0, 4)
    dl = O.token_logprobs_backward(logits, t, 1.0, f64(s.dlp), f64(s.dent))
    b = O.residual_norm_backward(dl @ p["head"], None, h, r, p["norm"], y, rp, p["post"], p["gate"], SCALE)
    want = {"head": dl.T @ out, "norm": b["dweight"], "post": b["dpost_weight"], "gate": b["dgate"].sum(0),
            "w": b["dy"].T @ x}
    near = lambda got, w: np.linalg.norm(f64(got) - w) <= 0.05 * np.linalg.norm(w)
    for k, v in want.items():
        assert near(s.g[k], v), k
    assert near(s.dx, b["dresidual"])
    # logits of about 2 in bf16, after two rounded tensors: a few hundredths each
    assert np.abs(f64(s.lp) - o["logprob"]).max() <= 0.1 and np.abs(f64(s.ent) - o["entropy"]).max() <= 0.1


@pytest.mark.parametrize("state_bits", [32, 8])
def test_steps(gpu_lib, state_bits):
    """Three steps: each parameter is, bit for bit, AdamW's of the gradient and states that the step had."""
    s = Step(gpu_lib, state_bits)
    for t in (1, 2, 3):
        before = {k: (v.clone(), [x.clone() if isinstance(x, torch.Tensor) else [q.clone() for q in x]
                                  for x in s.states[k]]) for k, v in s.master.items()}
        s.step(t)
        torch.cuda.synchronize()
        for k, (p, st) in before.items():
            n = p.numel()
            host = lambda q: q.view(torch.uint8).cpu().numpy() if q.dtype == torch.float8_e4m3fn else q.cpu().numpy()
            if state_bits == 8:
                st = [O.state_read(host(c), host(x), 256, i + 1).astype(np.float32) for i, (c, x) in enumerate(st)]
            else:
                st = [x.cpu().numpy() for x in st]
            want, _, _ = O.adamw(p.cpu().numpy().reshape(n), s.g[k].float().cpu().numpy().reshape(n), *st, step=t,
                                 weight_decay=0.1 if k in ("w", "head") else 0.0, **HP)
            assert np.array_equal(s.master[k].cpu().numpy().reshape(n), want), (k, t)
            assert torch.equal(s.p[k], s.master[k].to(BF)), (k, t)


def test_a_captured_step_is_the_eager_one(gpu_lib):
    """The whole step captured and replayed, with eager steps of another copy between; the hyper-parameters are
    those of the capture."""
    a, b = Step(gpu_lib, 8), Step(gpu_lib, 8)
    a.step(1)
    b.step(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(2)
    for i in range(3):
        graph.replay()
        b.step(2)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.results(), b.results())), i
