"""The training operators as a training step runs them: norm, router, rows to the
experts and back, norm, head loss, the way back through all of them, gradient
clipping and AdamW with 8-bit states, against torch's float64 autograd on the CPU;
and the step captured and replayed against the eager step on a stream of its own.

Bound of a gradient, in the norm of the tensor: a rounding to bf16 changes a value by
2^-8 of it at most, and a tensor by as much in its norm.  Between a parameter and its
gradient lie at most 16 (x's norm, z, act(z), the experts' rows, y, y's norm; dz of the
head, dy's norm, dy, the rows' gradients, act's, its product, their sum, dlogits, the
norm's gradient, dx), each carried on by operators that do not enlarge a random error
against the value; together 16 * 2^-8.
"""
import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu
zs = None
DEV = "cuda:0"
T, H, E, K, FF, V = 150, 64, 16, 2, 96, 1003
R = T * K
EPS = 1e-5
CFG = dict(lr=1e-3, weight_decay=0.1, decoupled=True)
SHAPES = {"g1": (H,), "b1": (H,), "router": (H, E), "w1": (E, H, FF), "w2": (E, FF, H), "g2": (H,), "b2": (H,),
          "head": (V, H)}


def setup_module(module):
    global zs
    from fsdp_sharded_optimizer_shard_amd import zs as _zs
    zs = _zs


def empty(*shape, dtype=torch.bfloat16):
    return torch.full(shape, 5, dtype=dtype, device=DEV)


class Step:
    """The parameters, their states and every buffer of a step."""

    def __init__(self):
        g = torch.Generator().manual_seed(3)
        self.p, self.master, self.grad = {}, {}, {}
        for k, s in SHAPES.items():
            w = torch.randn(s, generator=g) * (s[-2] if k != "head" else H) ** -0.5 if len(s) > 1 else \
                torch.randn(s, generator=g) * 0.2 + (k[0] == "g")
            self.p[k] = w.to(torch.bfloat16).to(DEV)
            self.master[k] = self.p[k].float()
            self.grad[k] = empty(*s, dtype=torch.float32)
        n = [p.numel() for p in self.p.values()]
        self.m, self.v = ([torch.zeros(i, dtype=torch.uint8, device=DEV) for i in n] for _ in "mv")
        self.ms, self.vs = ([torch.zeros(-(-i // 32), dtype=torch.uint8, device=DEV) for i in n] for _ in "mv")
        self.tensors = zs.TensorList(list(self.master.values()), list(self.grad.values()), list(self.p.values()),
                                     self.m, self.v, self.ms, self.vs, decay=[len(s) > 1 for s in SHAPES.values()])
        self.x, self.targets = empty(T, H), torch.zeros(T, dtype=torch.int64, device=DEV)
        self.active, self.dloss = empty(T, dtype=torch.uint8), empty(T, dtype=torch.float32)
        self.router = zs.Router(E, K, groups=4, top_groups=2, scale=1.5)
        self.counter = torch.ones(1, dtype=torch.int64, device=DEV)
        self.table = zs.adam_table_device([zs.adam_cfg(step=t + 1, **CFG) for t in range(8)], DEV)
        f32 = torch.float32
        self.xn, self.logits, self.yn, self.y = empty(T, H), empty(T, E, dtype=f32), empty(T, H), empty(T, H)
        self.stats = empty(4, T, dtype=f32)
        self.experts, self.rows_of = empty(T, K, dtype=torch.int32), empty(T, K, dtype=torch.int32)
        self.weights, self.dweights = empty(T, K, dtype=f32), empty(T, K, dtype=f32)
        self.offsets = empty(E + 1, dtype=torch.int64)
        self.route_work = empty(max(1, zs.route_workspace(self.router, T)), dtype=torch.int32)
        self.xr, self.z, self.a, self.e = empty(R, H), empty(R, FF), empty(R, FF), empty(R, H)
        self.kept = zs.Saved(self.z, FF)
        self.loss, self.lse = empty(T, dtype=f32), empty(T, dtype=f32)
        self.work = empty(max(zs.linear_xent_workspace(T, V, H, b) for b in (False, True)), dtype=f32)
        self.norm_work = empty(zs.layer_norm_workspace(T, H), dtype=f32)
        self.dyn, self.dy, self.dx, self.dxn, self.dlogits = (empty(T, n) for n in (H, H, H, H, E))
        self.de, self.da, self.dxr = empty(R, H), empty(R, FF), empty(R, H)
        self.partials = empty(self.tensors.partials_count(), dtype=torch.float64)
        self.coef = empty(1, dtype=f32)

    def set(self, seed):
        """The step's tokens: padding at the end, which no expert and no loss sees."""
        g = torch.Generator().manual_seed(seed)
        pad = 7 + seed
        t = torch.randint(0, V, (T,), generator=g)
        t[T - pad:] = -100
        self.x.copy_(torch.randn(T, H, generator=g))
        self.targets.copy_(t)
        self.active.copy_((t >= 0).to(torch.uint8))
        self.dloss.fill_(1.0 / (T - pad))

    def run(self):
        p, g = self.p, self.grad
        m1, r1, m2, r2 = self.stats
        zs.layer_norm_forward(T, H, self.x, H, p["g1"], p["b1"], EPS, self.xn, H, m1, r1)
        zs.gemm_bf16(T, E, H, self.xn, H, zs.K_INNER, p["router"], E, zs.K_OUTER, self.logits, E, zs.FP32)
        zs.route_forward(self.router, T, self.logits, E, self.experts, self.weights, self.offsets, self.rows_of,
                         self.route_work, active=self.active)
        zs.experts_dispatch(T, K, H, self.xn, H, self.rows_of, R, self.xr, H)
        zs.gemm_grouped_rows_bf16(E, self.offsets, R, FF, H, self.xr, H, p["w1"], FF, zs.K_OUTER, H * FF, self.a, FF,
                                  zs.BF16, zs.Epilogue(act="silu", preact=self.kept))
        zs.gemm_grouped_rows_bf16(E, self.offsets, R, H, FF, self.a, FF, p["w2"], H, zs.K_OUTER, H * FF, self.e, H)
        zs.experts_combine(T, K, H, self.e, H, R, self.rows_of, self.y, H, self.weights, self.x, H)
        zs.layer_norm_forward(T, H, self.y, H, p["g2"], p["b2"], EPS, self.yn, H, m2, r2)
        zs.linear_xent_forward(T, V, H, self.yn, H, p["head"], H, zs.K_INNER, self.targets, self.loss, self.lse,
                               self.work)

        zs.linear_xent_backward(T, V, H, self.yn, H, p["head"], H, zs.K_INNER, self.targets, self.lse, self.dloss,
                                self.dyn, H, g["head"], H, 512, self.work)
        zs.layer_norm_backward(T, H, self.dyn, H, self.y, H, p["g2"], m2, r2, self.dy, H, g["g2"], g["b2"],
                               self.norm_work)
        zs.experts_combine_backward(T, K, H, self.dy, H, R, self.rows_of, self.weights, self.e, H, self.de, H,
                                    self.dweights)
        zs.gemm_grouped_depth_bf16(E, self.offsets, R, FF, H, self.a, FF, self.de, H, g["w2"], H, H * FF)
        zs.gemm_grouped_rows_bf16(E, self.offsets, R, FF, H, self.de, H, p["w2"], H, zs.K_INNER, H * FF, self.da, FF)
        zs.act_backward(R, FF, self.da, FF, "silu", self.kept, self.da, FF)
        zs.gemm_grouped_depth_bf16(E, self.offsets, R, H, FF, self.xr, H, self.da, FF, g["w1"], FF, H * FF)
        zs.gemm_grouped_rows_bf16(E, self.offsets, R, H, FF, self.da, FF, p["w1"], FF, zs.K_INNER, H * FF, self.dxr, H)
        zs.experts_combine(T, K, H, self.dxr, H, R, self.rows_of, self.dxn, H)
        zs.route_backward(self.router, T, self.logits, E, self.experts, self.dweights, self.dlogits, E)
        zs.gemm_saved_bf16(H, E, T, zs.Saved(self.xn, H), self.dlogits, E, g["router"], E)
        zs.gemm_bf16_epilogue(T, H, E, self.dlogits, E, zs.K_INNER, p["router"], E, zs.K_INNER, self.dxn, H, zs.BF16,
                              zs.Epilogue(residual=self.dxn, ldr=H))
        zs.layer_norm_backward(T, H, self.dxn, H, self.x, H, p["g1"], m1, r1, self.dx, H, g["g1"], g["b1"],
                               self.norm_work, residual=self.dy, ldr=H)

        zs.tensors_sumsq(self.tensors, self.partials)
        zs.clip_coef(self.partials, self.partials.numel(), 0.1, self.coef)
        zs.adam_tensors_table(self.tensors, self.table, 8, self.counter, seed=11, clip_coef=self.coef)
        zs.step_advance(self.counter)

    def results(self):
        out = {f"grad {k}": t for k, t in self.grad.items()}
        out.update({f"master {k}": t for k, t in self.master.items()})
        out.update({f"param {k}": t for k, t in self.p.items()})
        for k, l in (("m", self.m), ("v", self.v), ("ms", self.ms), ("vs", self.vs)):
            out.update({f"{k} {i}": t for i, t in enumerate(l)})
        out.update(loss=self.loss, dx=self.dx, experts=self.experts, rows=self.rows_of, counter=self.counter,
                   coef=self.coef)
        return out


def reference(step, experts):
    """Loss and gradients in float64, the experts of each token as given."""
    p = {k: t.double().cpu().requires_grad_() for k, t in step.p.items()}
    x = step.x.double().cpu().requires_grad_()
    xn = F.layer_norm(x, (H,), p["g1"], p["b1"], EPS)
    s = (xn @ p["router"]).softmax(-1)
    on = experts[:, 0] >= 0
    ids = experts.clamp(min=0).long()
    w = s.gather(1, ids)
    w = 1.5 * w / w.sum(1, keepdim=True) * on[:, None]
    y = x
    for j in range(K):
        a = F.silu(torch.einsum("th,thf->tf", xn, p["w1"][ids[:, j]]))
        y = y + w[:, j, None] * torch.einsum("tf,tfh->th", a, p["w2"][ids[:, j]])
    yn = F.layer_norm(y, (H,), p["g2"], p["b2"], EPS)
    t = step.targets.cpu()
    loss = F.cross_entropy(yn @ p["head"].T, t, ignore_index=-100, reduction="none")
    (loss * step.dloss.double().cpu()).sum().backward()
    return loss.detach(), {k: t.grad for k, t in p.items()}, x.grad, s.detach()


def test_step_against_float64():
    step = Step()
    step.set(0)
    before = {k: t.clone() for k, t in step.master.items()}
    start = {k: t.clone() for k, t in step.p.items()}
    step.run()
    torch.cuda.synchronize()
    experts = step.experts.cpu()
    after = step.p
    step.p = start
    loss, grads, dx, scores = reference(step, experts)
    step.p = after
    on = step.targets.cpu() >= 0
    assert (experts[~on] == -1).all() and (experts[on] >= 0).all()
    assert int(step.offsets[-1]) == K * int(on.sum())
    # a choice may differ from float64's between scores that the roundings of x's norm
    # leave equal: the chosen are within 2^-5 of the best of their groups
    s = scores[on]
    assert (s.gather(1, experts[on][:, :1].long())[:, 0] >= s.max(1).values * (1 - 2.0 ** -5)).all()
    bound = 16 * 2.0 ** -8

    def near(got, want, what):
        e = float((got.double().cpu() - want).norm() / want.norm())
        assert e <= bound, (what, e)
    near(step.loss, loss, "loss")
    assert not step.loss.cpu()[~on].any()
    near(step.dx, dx, "dx")
    for k in SHAPES:
        near(step.grad[k], grads[k], k)

    # the clip and the first AdamW step, from the step's own gradients
    norm = sum(float((g.double() ** 2).sum()) for g in step.grad.values()) ** 0.5
    coef = min(1.0, 0.1 / (norm + 1e-6))
    assert coef < 1 and abs(float(step.coef) / coef - 1) < 2.0 ** -20
    for k, s in SHAPES.items():
        g = step.grad[k].double() * coef
        lr, wd = CFG["lr"], CFG["weight_decay"] if len(s) > 1 else 0.0
        want = before[k].double() * (1 - lr * wd) - lr * g / (g.abs() + 1e-8)
        # scalars and operations in fp32, the quotient within 2^-20; |g| near the 1e-8
        # of the divisor, or its square near fp32's least, makes it no worse
        assert ((step.master[k].double() - want).abs() <= lr * 2.0 ** -17 + want.abs() * 2.0 ** -22).all(), k
        assert torch.equal(step.p[k], step.master[k].to(torch.bfloat16))


def test_replayed_step_has_the_eager_steps_bits():
    """A captured step replayed with other tokens each time, eager steps of other buffers
    on a stream of their own between the replays."""
    a, b = Step(), Step()
    side = torch.cuda.Stream()
    a.set(0)
    b.set(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for t in range(4):
        a.set(t)
        graph.replay()
        with torch.cuda.stream(side):
            b.set(t)
            b.run()
        torch.cuda.synchronize()
        want = b.results()
        for k, v in a.results().items():
            assert torch.equal(v, want[k]), (t, k)
    assert int(a.counter) == 5
