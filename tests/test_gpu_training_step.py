"""The operators of a training step together, as a stack uses them: the shards of a
vocabulary looked up and added by the allreduce, dropout and a layer norm, a block
whose ranks' partial products meet in residual_dropout, the router with its balance
loss, a last norm, and all gradients back into the tables, against a plain 64-bit
form by autograd. One run is eager, on a stream of its own; another is captured into
a CUDA graph with its own buffers and replayed."""
import numpy as np
import pytest
import torch

import precision_collective_reduction_gb300 as pcr
import training_ref as ref

pytestmark = pytest.mark.gpu
RANKS, V, T, H, E, K = 2, 37, 90, 68, 8, 2
P, COEF, EPS = 0.25, 0.5, float(np.float32(1e-5))


class Step:
    """Weights, inputs and buffers of one step, and the step itself."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, device="cuda", generator=g) * scale

        def empty(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device="cuda")
        self.tables = [normal(V, H) for _ in range(RANKS)]
        self.ids = torch.randint(-2, RANKS * V + 2, (T,), device="cuda", generator=g)
        self.ids[5:25] = 3
        self.valid = torch.ones(T, dtype=torch.uint8, device="cuda")
        self.valid[80:] = 0
        self.w = [1 + normal(H, scale=0.2) for _ in range(2)]
        self.b = [normal(H, scale=0.2) for _ in range(2)]
        self.products = [normal(H, H, scale=H ** -0.5) for _ in range(RANKS)]
        self.router = normal(H, E, scale=H ** -0.5)
        self.rng = [torch.tensor([11, i], device="cuda") for i in range(2)]
        self.dy, self.dweights, self.dloss = normal(T, H), normal(T, K), normal(1)
        self.parts = [empty(T, H) for _ in range(RANKS)]
        self.sums = [empty(T, H) for _ in range(RANKS)]
        self.x0, self.n0, self.x1, self.n1, self.y = (empty(T, H) for _ in range(5))
        self.h = [empty(T, H) for _ in range(RANKS)]
        self.logits, self.dlogits = empty(T, E), empty(T, E)
        self.chosen, self.weights = empty(T, K, dtype=torch.int32), empty(T, K)
        self.loss, self.prob_sums = empty(1), empty(E)
        self.counts = empty(E + 1, dtype=torch.int32)
        self.dx1, self.dh, self.dx0, self.dsum, self.dn0 = (empty(T, H) for _ in range(5))
        self.dw = [empty(H) for _ in range(2)]
        self.db = [empty(H) for _ in range(2)]
        self.dtables = [empty(V, H) for _ in range(RANKS)]
        self.drouter, self.dproducts = empty(H, E), [empty(H, H) for _ in range(RANKS)]

    def run(self):
        for r in range(RANKS):
            pcr.token_embed(self.tables[r], self.ids, self.parts[r], first_id=r * V, scale=1.5)
        pcr.dda_flat_sim([p.view(-1) for p in self.parts], [s.view(-1) for s in self.sums], block=0)
        pcr.residual_dropout(self.sums[0], None, self.x0, self.rng[0], P, n_out=self.n0, w=self.w[0],
                             b=self.b[0], eps=EPS)
        for r in range(RANKS):
            torch.matmul(self.n0, self.products[r], out=self.h[r])
        pcr.residual_dropout(self.h, self.x0, self.x1, self.rng[1], P, n_out=self.n1, w=self.w[1],
                             b=self.b[1], eps=EPS)
        torch.matmul(self.n1, self.router, out=self.logits)
        pcr.expert_route(self.logits, self.chosen, self.weights)
        pcr.expert_balance(self.logits, self.chosen, self.loss, self.counts, self.prob_sums,
                           coef=COEF, valid=self.valid)
        pcr.layer_norm(self.n1, self.y, eps=EPS)
        # and back: y has the gradient dy, the weights dweights, the loss dloss
        pcr.expert_route_backward(self.logits, self.chosen, self.weights, self.dweights, self.dlogits)
        pcr.expert_balance_backward(self.logits, self.counts, self.dloss, self.dlogits, coef=COEF,
                                    valid=self.valid, accumulate=True)
        torch.matmul(self.n1.t(), self.dlogits, out=self.drouter)
        pcr.layer_norm_backward(self.dy, self.n1, self.dsum, eps=EPS)
        dn1 = torch.addmm(self.dsum, self.dlogits, self.router.t())
        pcr.residual_dropout_backward(None, dn1, self.x1, self.dx1, self.dh, self.rng[1], P,
                                      w=self.w[1], eps=EPS, dw=self.dw[1], db=self.db[1])
        torch.zeros(T, H, device="cuda", out=self.dn0)
        for r in range(RANKS):
            torch.matmul(self.n0.t(), self.dh, out=self.dproducts[r])
            self.dn0.addmm_(self.dh, self.products[r].t())
        pcr.residual_dropout_backward(self.dx1, self.dn0, self.x0, None, self.dx0, self.rng[0], P,
                                      w=self.w[0], eps=EPS, dw=self.dw[0], db=self.db[0])
        for r in range(RANKS):
            pcr.token_embed_backward(self.dx0, self.ids, self.dtables[r], first_id=r * V, scale=1.5)

    def results(self):
        return dict(x0=self.x0, n0=self.n0, x1=self.x1, n1=self.n1, y=self.y, loss=self.loss,
                    weights=self.weights, drouter=self.drouter, dw0=self.dw[0], dw1=self.dw[1],
                    db0=self.db[0], db1=self.db[1],
                    **{"dtable%d" % r: t for r, t in enumerate(self.dtables)},
                    **{"dproduct%d" % r: t for r, t in enumerate(self.dproducts)})

    def plain(self):
        """The same in 64 bits, given the experts that were chosen."""
        def leaf(t):
            return t.double().requires_grad_()
        tables, products = [leaf(t) for t in self.tables], [leaf(t) for t in self.products]
        w, b, router = [leaf(t) for t in self.w], [leaf(t) for t in self.b], leaf(self.router)
        keep = [torch.from_numpy(ref.kept(T, H, 11, i, P)).cuda() / (1 - P) for i in range(2)]

        def norm(x):
            d = x - x.mean(1, keepdim=True)
            return d / (d.square().mean(1, keepdim=True) + EPS).sqrt()
        x0 = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for r, table in enumerate(tables):
            at = torch.nonzero((self.ids >= r * V) & (self.ids < (r + 1) * V))[:, 0]
            x0 = x0.index_add(0, at, 1.5 * table[self.ids[at] - r * V])
        x0 = x0 * keep[0]
        n0 = norm(x0) * w[0] + b[0]
        x1 = x0 + sum(n0 @ m for m in products) * keep[1]
        n1 = norm(x1) * w[1] + b[1]
        p = torch.softmax(n1 @ router, 1)
        weights = p.gather(1, self.chosen.long())
        some = self.valid != 0
        n = torch.bincount(self.chosen[some].reshape(-1).long(), minlength=E).double()
        loss = (COEF * E * (n / n.sum() * p[some].mean(0)).sum()).view(1)
        y = norm(n1)
        torch.autograd.backward([y, weights, loss], [self.dy.double(), self.dweights.double(),
                                                     self.dloss.double()])
        return dict(x0=x0, n0=n0, x1=x1, n1=n1, y=y, loss=loss, weights=weights,
                    drouter=router.grad, dw0=w[0].grad, dw1=w[1].grad, db0=b[0].grad,
                    db1=b[1].grad, **{"dtable%d" % r: t.grad for r, t in enumerate(tables)},
                    **{"dproduct%d" % r: t.grad for r, t in enumerate(products)})


def check(step):
    got, want = step.results(), step.plain()
    assert torch.equal(step.counts[:E], torch.bincount(
        step.chosen[step.valid != 0].reshape(-1).long(), minlength=E).int())
    # FP32 products of 68 and 90 terms and norms in a chain of ten operators: 10 * 90 *
    # 2^-24 of the sums' magnitudes, which are some ten times the results': 1e-3 of the
    # norm leaves room, a wrong term does not pass
    for name, t in got.items():
        w = want[name].detach()
        assert float((t.double() - w).norm()) <= 1e-3 * float(w.norm()) + 1e-9, name


@pytest.fixture(autouse=True)
def full_precision():
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = old


def test_step_against_64_bits_on_another_stream():
    step = Step(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step.run()
    s.synchronize()
    check(step)


def test_captured_steps_that_take_turns_with_an_eager_one():
    # two graphs, captured one after the other, and eager calls between their replays:
    # none may meet the others' scratch memory
    steps = [Step(2), Step(3), Step(4)]
    for step in steps:
        step.run()
    torch.cuda.synchronize()
    want = [{k: t.clone() for k, t in step.results().items()} for step in steps]
    graphs = []
    for step in steps[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step.run()
        graphs.append(g)
    for step in steps:
        for t in step.results().values():
            t.fill_(7.0)
    for _ in range(3):
        for g in graphs:
            g.replay()
        steps[2].run()
    torch.cuda.synchronize()
    for step, w in zip(steps, want):
        for k, t in step.results().items():
            # the library's own results bit for bit; torch's products may take another way
            assert torch.allclose(t, w[k], rtol=1e-4, atol=1e-5), k
    check(steps[0])
    check(steps[2])
