"""The few-token expert layer against its definition in 64 bits (gpu).

Tolerances: a product's accumulation may truncate, 2^-23 of the running sum an
addition, over a chain of at most n / 32 + 32 additions (a warp's share of the
axis, its lanes, the warps' partial sums); the activation adds a few fp32
steps; as the sum of two values of the type it is off by the square of the
type's half step (fp16: no less than 2^-25); the output by half a step."""
import pytest
import torch

from moe_expert_epilogue_b200 import _abi, ops

pytestmark = pytest.mark.gpu

bf, hf, f32 = torch.bfloat16, torch.float16, torch.float32
HALF = {bf: 2.0 ** -8, hf: 2.0 ** -11}
INF = float("inf")


def _inputs(tokens, hidden, inter, experts, dt, dev, seed=0, router_dt=None):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    return {"x": r(tokens, hidden).to(dt),
            "w1": (r(experts, 2 * inter, hidden) * 1.5 * hidden ** -0.5).to(dt),
            "w2": (r(experts, hidden, inter) * max(inter, 1) ** -0.5).to(dt),
            "router_weight": (r(experts, hidden) * hidden ** -0.5).to(router_dt or dt),
            "shared_expert_output": r(tokens, hidden).to(dt), "residual": r(tokens, hidden).to(dt)}


def _acc(n):
    return (n / 32 + 32) * 2.0 ** -23


def _reference(x, w1, w2, ids, weights, limit, shared=None, residual=None):
    """(out, tolerance) in 64 bits, for the choice given."""
    dt = x.dtype
    x, inter = x.double(), w2.shape[2]
    out = torch.zeros_like(x)
    tol = torch.zeros_like(x)
    big = torch.zeros_like(x)
    half = HALF[dt]
    tiny = 2.0 ** -25 if dt == hf else 0.0
    for e in range(w1.shape[0]):
        t, k = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        a, b = w1[e].double().t(), w2[e].double().t()
        z, ez = x[t] @ a, (x[t].abs() @ a.abs()) * _acc(x.shape[1])
        p = weights[t, k].double()[:, None]
        g, u = z[:, :inter].clamp(max=limit), z[:, inter:].clamp(-limit, limit)
        s = torch.nn.functional.silu(g)
        h = p * s * u
        # |silu'| <= 1.1
        eh = p.abs() * (1.1 * u.abs() * ez[:, :inter] + (s.abs() + 1.1 * ez[:, :inter])
                        * ez[:, inter:]) + h.abs() * (16 * 2.0 ** -24 + half * half) + tiny
        y = h @ b
        out.index_add_(0, t, y)
        big.index_add_(0, t, y.abs())
        tol.index_add_(0, t, eh @ b.abs() + (h.abs() @ b.abs()) * _acc(inter))
    for other in (shared, residual):
        if other is not None:
            out = out + other.double()
            big = big + other.double().abs()
    tiny_out = 2.0 ** -25 if dt == hf else 2.0 ** -134
    return out, tol + big * (ids.shape[1] + 2) * 2.0 ** -24 + half * out.abs() + tiny_out


def _run(d, top_k, limit=INF, logits=None, **kw):
    t = d["x"].shape[0]
    dev = d["x"].device
    w = torch.full((t, top_k), 7.0, device=dev)
    ids = torch.full((t, top_k), 99, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    args = dict(d)
    if logits is not None:
        args["logits"], args["router_weight"] = logits, None
    args.update(kw)
    out = ops.moe_layer_small_batch(args.pop("x"), args.pop("w1"), args.pop("w2"), top_k,
                                    limit=limit, topk_weights=w, topk_ids=ids, dev_err=err, **args)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out, w, ids


def _expected_choice(d, top_k, logits=None, **kw):
    if logits is None:
        logits = (d["x"].double() @ d["router_weight"].double().t()).float()
    return ops.router_topk_fwd(logits, top_k, **kw)


def _compare(d, out, w, ids, limit, shared=True, residual=True):
    want, tol = _reference(d["x"], d["w1"], d["w2"], ids, w, limit,
                           d["shared_expert_output"] if shared else None,
                           d["residual"] if residual else None)
    bad = ~((out.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), out[bad][:4], want[bad][:4], tol[bad][:4])


# tokens, hidden, inter, experts, top_k: aligned and odd widths, one token to the most, units
# cut at 32 tokens, widths around the kernels' chunks of 256 and 1024
SIZES = [(1, 64, 64, 4, 2), (1, 1024, 512, 8, 8), (1, 4096, 1024, 16, 4), (2, 264, 136, 5, 3),
         (3, 7, 5, 3, 2), (5, 129, 33, 9, 4), (8, 1000, 520, 12, 6), (9, 2056, 256, 33, 8),
         (13, 1224, 616, 60, 6), (16, 512, 1032, 8, 2), (31, 96, 40, 300, 10), (33, 256, 256, 1, 1),
         (64, 768, 384, 4, 4), (100, 321, 70, 6, 5), (128, 512, 256, 64, 8), (128, 136, 72, 2, 1),
         (128, 64, 16, 512, 8), (32, 128, 24, 64, 32), (4, 2048, 2048, 8, 2)]


@pytest.mark.parametrize("dt", [bf, hf])
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", SIZES)
def test_sizes(cuda_device, tokens, hidden, inter, experts, top_k, dt):
    d = _inputs(tokens, hidden, inter, experts, dt, cuda_device, seed=tokens + hidden)
    out, w, ids = _run(d, top_k, limit=2.0)
    ew, eids = _expected_choice(d, top_k)
    assert torch.equal(ids, eids) and torch.equal(w, ew)
    _compare(d, out, w, ids, 2.0)


@pytest.mark.parametrize("score", [ops.MOE_SCORE_SOFTMAX, ops.MOE_SCORE_SIGMOID])
@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("router_dt", [bf, f32])
def test_router_modes(cuda_device, score, normalise, router_dt):
    d = _inputs(17, 520, 136, 40, bf, cuda_device, seed=3, router_dt=router_dt)
    kw = dict(score=score, normalise=normalise, scale=1.5)
    out, w, ids = _run(d, 5, limit=7.0, **kw)
    ew, eids = _expected_choice(d, 5, **kw)
    assert torch.equal(ids, eids) and torch.equal(w, ew)
    _compare(d, out, w, ids, 7.0)


@pytest.mark.parametrize("ldt", [f32, bf, hf])
def test_given_logits_and_closed_experts(cuda_device, ldt):
    """The caller's logits: closed experts (-inf), tokens with fewer open experts than choices,
    and one with none, whose row is the residual and the shared output alone."""
    d = _inputs(12, 256, 128, 20, bf, cuda_device, seed=5)
    g = torch.Generator(device=cuda_device).manual_seed(6)
    logits = torch.randn(12, 20, generator=g, device=cuda_device)
    logits[torch.rand(12, 20, generator=g, device=cuda_device) < 0.4] = -INF
    logits[3] = -INF
    logits[4] = -INF
    logits[4, 19] = 1.0
    logits = logits.to(ldt)
    out, w, ids = _run(d, 6, logits=logits)
    ew, eids = _expected_choice(d, 6, logits)
    assert torch.equal(ids, eids) and torch.equal(w, ew)
    assert (ids[3] == -1).all() and ids[4].tolist() == [19, -1, -1, -1, -1, -1]
    _compare(d, out, w, ids, INF)
    none = torch.full_like(logits, -INF)
    out, w, ids = _run(d, 6, logits=none)
    assert (ids == -1).all() and (w == 0).all()
    want = d["residual"].float() + d["shared_expert_output"].float()
    assert torch.equal(out, want.to(bf))


@pytest.mark.parametrize("tokens", [40, 100])
def test_all_tokens_on_the_same_experts(cuda_device, tokens):
    """More tokens of an expert than one unit holds."""
    d = _inputs(tokens, 264, 264, 10, bf, cuda_device, seed=7)
    logits = torch.arange(10, device=cuda_device).float().repeat(tokens, 1)
    out, w, ids = _run(d, 3, logits=logits, limit=5.0)
    assert (ids == torch.tensor([9, 8, 7], device=cuda_device)).all()
    _compare(d, out, w, ids, 5.0)


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("residual", [True, False])
def test_optional_terms_and_in_place(cuda_device, shared, residual):
    d = _inputs(6, 512, 64, 8, bf, cuda_device, seed=9)
    kw = {}
    if not shared:
        kw["shared_expert_output"] = None
    if not residual:
        kw["residual"] = None
    out, w, ids = _run(d, 2, **kw)
    _compare(d, out, w, ids, INF, shared, residual)
    if residual:
        r = d["residual"].clone()
        out2, _, _ = _run(d, 2, **{**kw, "residual": r, "out": r})
        assert out2.data_ptr() == r.data_ptr() and torch.equal(r, out)


@pytest.mark.parametrize("dt", [bf, hf])
@pytest.mark.parametrize("hidden,inter", [(512, 192), (1001, 75)])
def test_a_token_does_not_depend_on_the_others(cuda_device, hidden, inter, dt):
    """The same bits alone, in a small batch and in a full one, and run after run."""
    d = _inputs(128, hidden, inter, 16, dt, cuda_device, seed=11)
    out, w, ids = _run(d, 4, limit=7.0)
    for _ in range(2):
        assert torch.equal(_run(d, 4, limit=7.0)[0], out)
    for n in (1, 2, 7, 31, 64):
        part = {k: (v[5:5 + n] if k in ("x", "shared_expert_output", "residual") else v)
                for k, v in d.items()}
        o, wn, idn = _run(part, 4, limit=7.0)
        assert torch.equal(idn, ids[5:5 + n]) and torch.equal(wn, w[5:5 + n])
        assert torch.equal(o, out[5:5 + n])


@pytest.mark.parametrize("valid", [0, 1, 9, 16, -3, 17])
def test_valid_tokens(cuda_device, valid):
    d = _inputs(16, 264, 72, 6, bf, cuda_device, seed=13)
    full, w, ids = _run(d, 3)
    n = torch.tensor([valid], dtype=torch.int32, device=cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = torch.full_like(full, 5.0)
    w2, ids2 = torch.full_like(w, 7.0), torch.full_like(ids, 99)
    live = min(max(valid, 0), 16)
    x = d["x"].clone()
    x[live:] = float("nan")                  # the padding's contents do not matter
    ops.moe_layer_small_batch(x, d["w1"], d["w2"], 3, router_weight=d["router_weight"],
                              shared_expert_output=d["shared_expert_output"],
                              residual=d["residual"], valid_tokens=n, out=out, topk_weights=w2,
                              topk_ids=ids2, dev_err=err)
    assert torch.equal(out[:live], full[:live]) and (out[live:] == 5).all()
    assert torch.equal(w2[:live], w[:live]) and (w2[live:] == 7).all()
    assert torch.equal(ids2[:live], ids[:live]) and (ids2[live:] == 99).all()
    assert int(err) == (_abi.MOE_DEVERR_COUNT if valid in (-3, 17) else 0)


@pytest.mark.parametrize("hidden,inter", [(520, 136), (515, 67)])
def test_strides_and_alignment(cuda_device, hidden, inter):
    """x, shared, residual and out inside wider buffers, weights off a 16-byte boundary: the
    same bits, and what lies between the rows stays."""
    t, e = 10, 7
    d = _inputs(t, hidden, inter, e, bf, cuda_device, seed=15)
    want, _, _ = _run(d, 3, limit=7.0)
    for offset, pad in ((0, 8), (1, 3), (2, 0)):
        def inside(v, fill=3.0):
            buf = torch.full((offset + t * (hidden + pad),), fill, dtype=bf, device=cuda_device)
            s = buf[offset:].view(t, hidden + pad)[:, :hidden]
            if v is not None:
                s.copy_(v)
            return buf, s

        def shifted(w):
            buf = torch.empty(offset + w.numel(), dtype=bf, device=cuda_device)
            v = buf[offset:].view(w.shape)
            v.copy_(w)
            return v

        moved = {k: shifted(d[k]) for k in ("w1", "w2", "router_weight")}
        moved.update({k: inside(d[k])[1] for k in ("x", "shared_expert_output", "residual")})
        buf, o = inside(None)
        out, _, _ = _run(moved, 3, limit=7.0, out=o)
        assert torch.equal(o, want)
        assert (buf[:offset] == 3).all()
        assert (buf[offset:].view(t, hidden + pad)[:, hidden:] == 3).all()


def test_no_tokens_no_columns(cuda_device):
    d = _inputs(0, 64, 32, 4, bf, cuda_device)
    assert _run(d, 2)[0].shape == (0, 64)
    d = _inputs(3, 64, 0, 4, bf, cuda_device)
    out, _, _ = _run(d, 2)
    want = d["residual"].float() + d["shared_expert_output"].float()
    assert torch.equal(out, want.to(bf))


def test_large_and_non_finite_activations(cuda_device):
    """fp16 activations beyond 65504 are carried by their two halves; an infinite one stays
    infinite, and NaN stays with its token."""
    d = _inputs(4, 64, 16, 2, hf, cuda_device, seed=17)
    d["w1"].fill_(2.0)
    d["w2"].fill_(2.0 ** -10)
    d["x"].fill_(2.34375)                    # z = 300, h = 300 * 300 = 90000
    logits = torch.tensor([[0.0, -INF]], device=cuda_device).repeat(4, 1)
    d["residual"].zero_()
    d["shared_expert_output"].zero_()
    d["x"][2, 0] = float("nan")
    out, _, _ = _run(d, 1, logits=logits)
    keep = [0, 1, 3]
    # 16 terms of 90000 * 2^-10: every sum is exact, and 1406.25 rounds to 1406
    assert (out[keep] == 1406).all()
    assert out[2].isnan().all()
    d["x"][2, 0] = INF
    out, _, _ = _run(d, 1, logits=logits)
    assert (out[2] == INF).all()


def test_workspace_streams_and_graphs(cuda_device):
    """A workspace full of anything, given or not; another stream; two captured graphs that
    share one workspace, replayed one after the other, as the counts and inputs change."""
    d = _inputs(9, 512, 136, 12, bf, cuda_device, seed=19)
    want, w, ids = _run(d, 4, limit=7.0)
    nbytes = ops.moe_layer_small_batch_workspace(9, 512, 136, 12, 4)
    for fill in (0, 0x7f, 0xff):
        ws = torch.full((nbytes,), fill, dtype=torch.uint8, device=cuda_device)
        assert torch.equal(_run(d, 4, limit=7.0, workspace=ws)[0], want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for handle in (s, s.cuda_stream):
        out, _, _ = _run(d, 4, limit=7.0, stream=handle)
        assert torch.equal(out, want)
    other = _inputs(3, 512, 136, 12, bf, cuda_device, seed=20)
    want2, _, _ = _run(other, 4)
    n = torch.tensor([9], dtype=torch.int32, device=cuda_device)
    out, out2 = torch.zeros_like(want), torch.zeros_like(want2)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        ops.moe_layer_small_batch(d["x"], d["w1"], d["w2"], 4, router_weight=d["router_weight"],
                                  limit=7.0, shared_expert_output=d["shared_expert_output"],
                                  residual=d["residual"], valid_tokens=n, out=out, workspace=ws)
    with torch.cuda.graph(graphs[1]):
        ops.moe_layer_small_batch(other["x"], other["w1"], other["w2"], 4,
                                  router_weight=other["router_weight"],
                                  shared_expert_output=other["shared_expert_output"],
                                  residual=other["residual"], out=out2, workspace=ws)
    for live in (9, 4):
        out.zero_()
        out2.zero_()
        n.fill_(live)
        for g in (graphs[0], graphs[1], graphs[0]):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:live], want[:live]) and (out[live:] == 0).all()
        assert torch.equal(out2, want2)


def test_two_streams_at_once(cuda_device):
    """Two calls in flight on two streams, each with its own workspace."""
    d = _inputs(16, 1024, 512, 16, bf, cuda_device, seed=21)
    want, _, _ = _run(d, 4)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(10):
        for s in (a, b):
            outs.append(ops.moe_layer_small_batch(
                d["x"], d["w1"], d["w2"], 4, router_weight=d["router_weight"],
                shared_expert_output=d["shared_expert_output"], residual=d["residual"], stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_the_block_of_a_decode_step(cuda_device):
    """Norm, router and layer of a step, as they run together: the layer's own router makes the
    choice that the router op makes of the same logits, and the next norm reads its output."""
    t, hid, inter, e, k = 6, 1024, 256, 16, 4
    d = _inputs(t, hid, inter, e, bf, cuda_device, seed=23)
    g = torch.Generator(device=cuda_device).manual_seed(24)
    nw = (1 + 0.1 * torch.randn(hid, generator=g, device=cuda_device)).to(bf)
    x, _, _ = ops.layer_norm_fwd(d["residual"], nw)
    logits = (x.double() @ d["router_weight"].double().t()).float()
    w, ids = ops.router_topk_fwd(logits, k)
    kw = dict(limit=7.0, shared_expert_output=d["shared_expert_output"], residual=d["residual"])
    a = ops.moe_layer_small_batch(x, d["w1"], d["w2"], k, router_weight=d["router_weight"], **kw)
    b = ops.moe_layer_small_batch(x, d["w1"], d["w2"], k, logits=logits, **kw)
    assert torch.equal(a, b)
    want, tol = _reference(x, d["w1"], d["w2"], ids, w, 7.0, d["shared_expert_output"],
                           d["residual"])
    assert ((a.double() - want).abs() <= tol).all()
    y, _, _ = ops.layer_norm_fwd(a, nw)
    assert y.isfinite().all()
    # the same step through the ops of the many-token path, expert rows by the library product
    rows = torch.zeros(t * k, hid, dtype=bf, device=cuda_device)
    order = ids.flatten().argsort(stable=True)
    inv = torch.full((t, e), -1, dtype=torch.int32, device=cuda_device)
    for r, slot in enumerate(order.tolist()):
        ei = int(ids.flatten()[slot])
        act = ops.swiglu_clamped_fwd(x[slot // k][None] @ d["w1"][ei].t(),
                                     w.flatten()[slot].view(1, 1), 7.0)
        rows[r] = (act @ d["w2"][ei].t())[0]
        inv[slot // k, ei] = r
    n = torch.tensor([t], dtype=torch.int32, device=cuda_device)
    many = ops.epilogue_fused(rows, torch.ones(t * k, device=cuda_device), inv, n,
                              d["shared_expert_output"], d["residual"])
    # that path rounds to bf16 at the products, the activation, each row, the sum and the output
    scale = want.abs() + d["shared_expert_output"].double().abs() + d["residual"].double().abs() + 2
    assert ((a.double() - many.double()).abs() <= 8 * 2.0 ** -8 * scale).all()


@pytest.mark.parametrize("tokens", [3, 30])
def test_captured_before_any_eager_call_of_its_shape(cuda_device, tokens):
    """A graph whose capture is the first call of these sizes; two replays of it in flight on
    one stream behind changing inputs."""
    d = _inputs(tokens, 712, 88, 24, bf, cuda_device, seed=31)
    ws = torch.empty(ops.moe_layer_small_batch_workspace(tokens, 712, 88, 24, 5),
                     dtype=torch.uint8, device=cuda_device)
    out = torch.zeros(tokens, 712, dtype=bf, device=cuda_device)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.moe_layer_small_batch(d["x"], d["w1"], d["w2"], 5, router_weight=d["router_weight"],
                                  residual=d["residual"], out=out, workspace=ws)
    x0 = d["x"].clone()
    g.replay()
    first = out.clone()
    d["x"].neg_()
    g.replay()
    second = out.clone()
    d["x"].copy_(x0)
    kw = dict(router_weight=d["router_weight"], residual=d["residual"])
    assert torch.equal(first, ops.moe_layer_small_batch(x0, d["w1"], d["w2"], 5, **kw))
    assert torch.equal(second, ops.moe_layer_small_batch(-x0, d["w1"], d["w2"], 5, **kw))


@pytest.mark.parametrize("fill", ["nan", "inf"])
def test_a_bad_token_stays_with_itself(cuda_device, fill):
    """A token whose input is not finite spoils its own row alone."""
    d = _inputs(20, 520, 136, 9, bf, cuda_device, seed=33)
    logits = torch.randn(20, 9, device=cuda_device,
                         generator=torch.Generator(device=cuda_device).manual_seed(34))
    want, _, _ = _run(d, 3, logits=logits)
    d["x"][7] = float(fill)
    got, _, _ = _run(d, 3, logits=logits)
    keep = [t for t in range(20) if t != 7]
    assert torch.equal(got[keep], want[keep]) and not got[7].isfinite().any()


def test_weights_past_32_bits(cuda_device):
    """Experts whose weights start beyond 2^31 elements."""
    e, inter, hid = 400, 2048, 2112
    d = _inputs(2, hid, 8, 1, bf, cuda_device, seed=35)
    w1 = torch.empty(e, 2 * inter, hid, dtype=bf, device=cuda_device)
    w2 = torch.empty(e, hid, inter, dtype=bf, device=cuda_device)
    assert w1.numel() > 2 ** 31 and w1.numel() + w2.numel() > 2 ** 32
    g = torch.Generator(device=cuda_device).manual_seed(36)
    for i in (0, e - 1):
        w1[i] = (torch.randn(2 * inter, hid, generator=g, device=cuda_device) * hid ** -0.5).to(bf)
        w2[i] = (torch.randn(hid, inter, generator=g, device=cuda_device) * inter ** -0.5).to(bf)
    logits = torch.full((2, e), -INF, device=cuda_device)
    logits[0, e - 1] = 1.0
    logits[1, 0], logits[1, e - 1] = 0.5, 0.25
    out = ops.moe_layer_small_batch(d["x"], w1, w2, 2, logits=logits, residual=d["residual"])
    small1, small2 = w1[[0, e - 1]].contiguous(), w2[[0, e - 1]].contiguous()
    want = ops.moe_layer_small_batch(d["x"], small1, small2, 2,
                                     logits=logits[:, [0, e - 1]].contiguous(),
                                     residual=d["residual"])
    assert torch.equal(out, want)


# tokens, hidden, inter, experts, top_k of narrow, wide and odd tiles: at least three fills of the
# first CTA in either product
STALLS = [("narrow", 2, 4096, 1024, 4, 2), ("wide", 40, 2048, 1024, 8, 4),
          ("odd", 30, 2047, 515, 8, 4)]


@pytest.mark.parametrize("stall", range(6))
@pytest.mark.parametrize("tiles,tokens,hidden,inter,experts,top_k", STALLS)
def test_bounded_waits_run_out(cuda_device, tiles, tokens, hidden, inter, experts, top_k, stall):
    """The first CTA withholds a stage of weights (first or second product), a stage of tokens or
    an arrival at a grid barrier: the waits give up after 2e7 cycles (10 ms), the producers stop,
    the copies issued are waited for and the call ends with MOE_DEVERR_TIMEOUT.  The next ordinary
    calls, on the same workspace, have their bits."""
    if stall == 3 and tokens <= 24:
        pytest.skip("every CTA makes the choice for itself")
    d = _inputs(tokens, hidden, inter, experts, bf, cuda_device, seed=41)
    g = torch.Generator(device=cuda_device).manual_seed(42)
    logits = torch.randn(tokens, experts, generator=g, device=cuda_device)
    ws = torch.empty(ops.moe_layer_small_batch_workspace(tokens, hidden, inter, experts, top_k),
                     dtype=torch.uint8, device=cuda_device)
    kw = dict(logits=logits, shared_expert_output=None, residual=None, workspace=ws)
    want, _, _ = _run(d, top_k, **kw)
    _abi.moe_device_errors(clear=True)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = torch.zeros_like(want)
    _abi.moe_test_layer_small_batch_stalled(d["x"], logits, d["w1"], d["w2"], out, ws, ws.numel(),
                                            tokens, hidden, inter, experts, top_k, stall,
                                            20_000_000, err)
    torch.cuda.synchronize()
    assert int(err) == _abi.MOE_DEVERR_TIMEOUT
    assert _abi.moe_device_errors(clear=True) == 0
    for _ in range(2):
        assert torch.equal(_run(d, top_k, **kw)[0], want)


@pytest.mark.parametrize("inter", [0, 24])
@pytest.mark.parametrize("tokens", [3, 70])
def test_the_choice_without_columns(cuda_device, tokens, inter):
    """A hidden axis of no columns: the choice is made all the same, of the logits given or, with
    a router of no columns, of logits 0."""
    e = lambda *shape: torch.empty(*shape, dtype=bf, device=cuda_device)  # noqa: E731
    d = {"x": e(tokens, 0), "w1": e(9, 2 * inter, 0), "w2": e(9, 0, inter),
         "router_weight": e(9, 0), "shared_expert_output": e(tokens, 0), "residual": e(tokens, 0)}
    g = torch.Generator(device=cuda_device).manual_seed(43)
    logits = torch.randn(tokens, 9, generator=g, device=cuda_device)
    logits[1] = -INF
    for z in (logits, None):
        out, w, ids = _run(d, 4, logits=z)
        ew, eids = ops.router_topk_fwd(torch.zeros_like(logits) if z is None else z, 4)
        assert out.shape == (tokens, 0) and torch.equal(ids, eids) and torch.equal(w, ew)


# More than 24 live tokens: the CTAs share the choices through the workspace, behind a grid barrier.


@pytest.mark.parametrize("tokens", [25, 40, 128])
@pytest.mark.parametrize("ldt", [f32, bf])
def test_shared_choices_of_closed_experts(cuda_device, tokens, ldt):
    """Closed experts, tokens with fewer open ones than choices and with none, over a workspace
    full of ones."""
    d = _inputs(tokens, 264, 72, 20, bf, cuda_device, seed=45)
    g = torch.Generator(device=cuda_device).manual_seed(46)
    logits = torch.randn(tokens, 20, generator=g, device=cuda_device)
    logits[torch.rand(tokens, 20, generator=g, device=cuda_device) < 0.5] = -INF
    logits[3::9] = -INF
    logits[4] = -INF
    logits[4, 19] = 1.0
    logits = logits.to(ldt)
    ws = torch.full((ops.moe_layer_small_batch_workspace(tokens, 264, 72, 20, 6),), 0xff,
                    dtype=torch.uint8, device=cuda_device)
    out, w, ids = _run(d, 6, logits=logits, workspace=ws)
    ew, eids = _expected_choice(d, 6, logits)
    assert torch.equal(ids, eids) and torch.equal(w, ew)
    assert (ids[3] == -1).all() and ids[4].tolist() == [19, -1, -1, -1, -1, -1]
    _compare(d, out, w, ids, INF)
    ws.fill_(0xff)
    out, w, ids = _run(d, 6, logits=torch.full_like(logits, -INF), workspace=ws)
    assert (ids == -1).all() and (w == 0).all()
    want = d["residual"].float() + d["shared_expert_output"].float()
    assert torch.equal(out, want.to(bf))


@pytest.mark.parametrize("score", [ops.MOE_SCORE_SOFTMAX, ops.MOE_SCORE_SIGMOID])
@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("tokens", [40, 128])
def test_shared_choices_router_modes(cuda_device, tokens, score, normalise):
    d = _inputs(tokens, 520, 136, 40, hf, cuda_device, seed=47)
    kw = dict(score=score, normalise=normalise, scale=1.5)
    out, w, ids = _run(d, 5, limit=7.0, **kw)
    ew, eids = _expected_choice(d, 5, **kw)
    assert torch.equal(ids, eids) and torch.equal(w, ew)
    _compare(d, out, w, ids, 7.0)


@pytest.mark.parametrize("tokens", [40, 128])
def test_valid_tokens_on_both_sides_of_the_shared_choice(cuda_device, tokens):
    """One captured graph as the count on the device goes up and down across 24."""
    d = _inputs(tokens, 264, 72, 6, bf, cuda_device, seed=48)
    full, w, ids = _run(d, 3)
    n = torch.tensor([tokens], dtype=torch.int32, device=cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    x, out = d["x"].clone(), torch.empty_like(full)
    w2, ids2 = torch.empty_like(w), torch.empty_like(ids)
    ws = torch.full((ops.moe_layer_small_batch_workspace(tokens, 264, 72, 6, 3),), 0xff,
                    dtype=torch.uint8, device=cuda_device)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_layer_small_batch(x, d["w1"], d["w2"], 3, router_weight=d["router_weight"],
                                  shared_expert_output=d["shared_expert_output"],
                                  residual=d["residual"], valid_tokens=n, out=out, topk_weights=w2,
                                  topk_ids=ids2, workspace=ws, dev_err=err)
    for valid in (tokens, 24, 25, 0, 39, 1, tokens + 1, 23, -3, 26):
        live = min(max(valid, 0), tokens)
        x.copy_(d["x"])
        x[live:] = float("nan")
        n.fill_(valid)
        err.zero_()
        for t, fill in ((out, 5.0), (w2, 7.0), (ids2, 99), (ws, 0xff)):
            t.fill_(fill)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:live], full[:live]) and (out[live:] == 5).all()
        assert torch.equal(w2[:live], w[:live]) and (w2[live:] == 7).all()
        assert torch.equal(ids2[:live], ids[:live]) and (ids2[live:] == 99).all()
        assert int(err) == (_abi.MOE_DEVERR_COUNT if valid != live else 0)


def test_two_streams_at_once_with_shared_choices(cuda_device):
    """Two calls of different shapes in flight on two streams, three grid barriers each."""
    d = [_inputs(40, 1024, 512, 16, bf, cuda_device, seed=49),
         _inputs(64, 768, 256, 8, bf, cuda_device, seed=50)]
    kw = [dict(router_weight=v["router_weight"], residual=v["residual"]) for v in d]
    want = [ops.moe_layer_small_batch(v["x"], v["w1"], v["w2"], 4, **k) for v, k in zip(d, kw)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [[ops.moe_layer_small_batch(v["x"], v["w1"], v["w2"], 4, stream=s, **k)
             for v, k, s in zip(d, kw, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for pair in outs for o, w in zip(pair, want))


@pytest.mark.parametrize("ldt", [f32, hf])
@pytest.mark.parametrize("tokens", [7, 50])
def test_logits_inside_a_wider_buffer(cuda_device, tokens, ldt):
    d = _inputs(tokens, 136, 40, 21, bf, cuda_device, seed=52)
    g = torch.Generator(device=cuda_device).manual_seed(53)
    wide = torch.randn(tokens, 30, generator=g, device=cuda_device).to(ldt) + 9
    part = wide[:, 5:26]
    got, want = _run(d, 4, logits=part), _run(d, 4, logits=part.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ew, eids = _expected_choice(d, 4, part)
    assert torch.equal(got[2], eids) and torch.equal(got[1], ew)
