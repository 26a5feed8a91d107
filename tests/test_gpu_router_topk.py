"""The top-k router and its gradient against their definitions in 64 bits (gpu).

Tolerances in u = 2^-24: an exponential is off by 2 u of its value beyond what
the rounded difference of its argument gives (u of the argument, at most 100
here before a term falls below 2^-126 of the largest), a sum of E terms by its
depth of at most E / 32 + 5 additions, a quotient and a product by u each."""
import pytest
import torch

from moe_expert_epilogue_b200 import ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
SOFT, SIG = ops.MOE_SCORE_SOFTMAX, ops.MOE_SCORE_SIGMOID
MODES = [(SOFT, True, 1.0), (SOFT, False, 1.0), (SIG, True, 2.5), (SIG, False, 0.5)]
INF = float("inf")


def _choose(logits, k):
    """Expert by expert: the largest logit left, the first of equals; -1 for none."""
    left = logits.double().cpu()
    ids = []
    for row in left:
        vals = [(-v, e) for e, v in enumerate(row.tolist()) if v != -INF]
        top = [e for _, e in sorted(vals)[:k]]
        ids.append(top + [-1] * (k - len(top)))
    return torch.tensor(ids, dtype=torch.int32, device=logits.device).reshape(-1, k)


def _weights(logits, ids, score, normalise, scale):
    z = logits.double()
    chosen = ids >= 0
    at = ids.long().clamp(min=0)
    if score == SOFT and normalise:
        w = torch.softmax(z.gather(1, at).masked_fill(~chosen, -INF), 1)
    elif score == SOFT:
        w = torch.softmax(z, 1).gather(1, at)
    else:
        w = torch.sigmoid(z).gather(1, at) * chosen
        if normalise:
            w = w / w.sum(1, keepdim=True)
    return torch.where(chosen, w * scale, torch.zeros_like(w))


def _tol(experts):
    return (experts / 32 + 5 + 200 + 8) * U


def _logits(tokens, experts, dt, seed, dev, masked=0.0, sigma=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    z = torch.randn(tokens, experts, generator=g, device=dev) * sigma
    if masked:
        z = z.masked_fill(torch.rand(tokens, experts, generator=g, device=dev) < masked, -INF)
    return z.to(dt), g


SIZES = [(1, 1, 1), (1, 8, 8), (3, 7, 2), (16, 64, 8), (5, 33, 4), (100, 60, 6), (9, 128, 8),
         (33, 161, 6), (40, 256, 8), (7, 300, 32), (5, 512, 9), (4, 1000, 8), (3, 1024, 32)]


@pytest.mark.parametrize("score,normalise,scale", MODES)
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("tokens,experts,top_k", SIZES)
def test_forward(cuda_device, tokens, experts, top_k, dt, score, normalise, scale):
    """bf16 and fp16 logits of many experts hold equal values: ties go to the lower expert."""
    z, _ = _logits(tokens, experts, dt, tokens + experts, cuda_device)
    w, ids = ops.router_topk_fwd(z, top_k, score, normalise, scale)
    assert torch.equal(ids, _choose(z, top_k))
    want = _weights(z, ids, score, normalise, scale)
    assert ((w.double() - want).abs() <= _tol(experts) * want.abs()).all()


@pytest.mark.parametrize("score,normalise,scale", MODES)
@pytest.mark.parametrize("dt", DTYPES)
def test_masked_experts(cuda_device, dt, score, normalise, scale):
    """-inf closes an expert; a row with fewer open experts than choices, with one, with none;
    rows of the type's lowest value."""
    z, _ = _logits(40, 64, dt, 3, cuda_device, masked=0.9)
    z[0] = -INF
    z[1] = -INF
    z[1, 63] = 0.25
    z[2] = torch.finfo(dt).min
    z[3] = -INF
    z[3, 5] = torch.finfo(dt).min
    z[4] = torch.finfo(dt).max
    w, ids = ops.router_topk_fwd(z, 8, score, normalise, scale)
    assert torch.equal(ids, _choose(z, 8))
    assert (ids[0] == -1).all() and ids[1].tolist() == [63] + [-1] * 7
    assert ids[2].tolist() == ids[4].tolist() == list(range(8))
    assert (w[ids < 0] == 0).all() and w.isfinite().all()
    want = _weights(z, ids, score, normalise, scale)
    if score == SIG and normalise:                  # 64 bits underflow as well there: by symmetry
        want[2], want[3] = scale / 8, torch.tensor([scale] + [0.0] * 7)
    want[0] = 0
    assert ((w.double() - want).abs() <= _tol(64) * want.abs()).all()


def test_zeros_of_both_signs_tie(cuda_device):
    z = torch.tensor([[-0.0, 0.0, -0.0, 0.0, -1.0]], device=cuda_device)
    assert ops.router_topk_fwd(z, 4)[1].tolist() == [[0, 1, 2, 3]]


def test_sigmoid_of_far_negative_logits(cuda_device):
    """sig(l) underflows in fp32 below -103, the quotients do not."""
    z = torch.tensor([[-200.0, -201.0, -300.0, -200.5]], device=cuda_device)
    w, ids = ops.router_topk_fwd(z, 3, SIG, True)
    want = torch.softmax(torch.tensor([-200.0, -200.5, -201.0], dtype=torch.float64), 0)
    assert ids.tolist() == [[0, 3, 1]]
    assert ((w[0].double().cpu() - want).abs() <= 300 * U * want).all()


def test_nan_and_infinity(cuda_device):
    z, _ = _logits(4, 64, torch.float32, 5, cuda_device)
    z[1, 7] = float("nan")
    z[2, 9] = INF
    w, ids = ops.router_topk_fwd(z, 8)
    assert ids[1, 0] == 7 and ids[2, 0] == 9
    assert w[1].isnan().all() and w[2].isnan().all() and w[[0, 3]].isfinite().all()
    clean = z.clone()
    clean[1:3] = 0
    w2, ids2 = ops.router_topk_fwd(clean, 8)
    assert torch.equal(w[[0, 3]], w2[[0, 3]]) and torch.equal(ids[[0, 3]], ids2[[0, 3]])


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("experts", [20, 64, 200, 400, 900])
def test_nan_of_either_sign_and_infinities_by_type(cuda_device, dt, experts):
    """NaN of either sign counts as the largest, whatever its bits; +inf comes next."""
    z, _ = _logits(6, experts, dt, 21, cuda_device)
    z[0, experts - 1] = float("nan")
    z[1, 3] = -torch.tensor(float("nan"))
    z[2, 5] = INF
    z[3, 1] = INF
    z[3, 7] = float("nan")
    z[4, :] = -INF
    z[4, 9] = -torch.tensor(float("nan"))
    _, ids = ops.router_topk_fwd(z, 2, SIG, False)
    assert ids[0, 0] == experts - 1 and ids[1, 0] == 3 and ids[2, 0] == 5
    assert ids[3].tolist() == [7, 1] and ids[4].tolist() == [9, -1]
    assert torch.equal(ids[5:], _choose(z[5:], 2))


def _exact_grad(z, ids, gw, score, normalise, scale):
    with torch.enable_grad():
        z = z.double().requires_grad_()
        g = torch.where(ids >= 0, gw.double(), torch.zeros_like(gw.double()))
        (gz,) = torch.autograd.grad((_weights(z, ids, score, normalise, scale) * g).sum(), z)
    return torch.nan_to_num(gz, nan=0.0)


@pytest.mark.parametrize("score,normalise,scale", MODES)
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("tokens,experts,top_k", SIZES)
def test_backward(cuda_device, tokens, experts, top_k, dt, score, normalise, scale):
    z, g = _logits(tokens, experts, dt, tokens, cuda_device, masked=0.1 if experts > 8 else 0.0)
    ids = ops.router_topk_fwd(z, top_k)[1]
    gw = torch.randn(tokens, top_k, generator=g, device=cuda_device)
    gl = ops.router_topk_bwd(z, ids, gw, score, normalise, scale)
    assert gl.dtype == dt
    want = _exact_grad(z, ids, gw, score, normalise, scale)
    # every term is a product of at most |scale g| and a share; the inner sum has top_k of them
    big = (gw.abs().amax(1, keepdim=True) * abs(scale)).double()
    share = _weights(z, torch.arange(experts, device=cuda_device, dtype=torch.int32).expand(
        tokens, experts), SOFT, False, 1.0) if score == SOFT and not normalise else \
        torch.zeros(tokens, experts, device=cuda_device, dtype=torch.float64).scatter_add(
            1, ids.long().clamp(min=0), _weights(z, ids, score, normalise, 1.0))
    tol = 2 * (_tol(experts) + top_k * U) * big * share + HALF[dt] * want.abs() + TINY[dt]
    assert ((gl.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("score,normalise,scale", MODES)
def test_backward_against_differences(cuda_device, score, normalise, scale):
    z, g = _logits(3, 12, torch.float32, 7, cuda_device)
    ids = ops.router_topk_fwd(z, 4)[1]
    gw = torch.randn(3, 4, generator=g, device=cuda_device)
    gl = ops.router_topk_bwd(z, ids, gw, score, normalise, scale)
    f = lambda z: float((_weights(z, ids, score, normalise, scale) * gw.double()).sum())  # noqa: E731
    for i in range(z.numel()):
        up, down = z.double().clone(), z.double().clone()
        up.view(-1)[i] += 1e-6
        down.view(-1)[i] -= 1e-6
        # 64-bit differences of step 1e-6: 1e-16 / 1e-6 of a sum of order 10, and 1e-12
        assert abs((f(up) - f(down)) / 2e-6 - float(gl.view(-1)[i])) <= 2e-6


@pytest.mark.parametrize("score,normalise,scale", MODES)
def test_backward_of_given_choices(cuda_device, score, normalise, scale):
    """Ids that no forward made: an empty slot's gradient is not read, an expert named twice gets
    both, an expert past the last is reported and skipped; every expert's column is written."""
    z, g = _logits(5, 40, torch.float32, 9, cuda_device)
    ids = torch.tensor([[3, -1, 7], [5, 5, 6], [-1, -1, -1], [39, 40, 2], [0, 1, 2]],
                       dtype=torch.int32, device=cuda_device)
    gw = torch.randn(5, 3, generator=g, device=cuda_device)
    gw[0, 1] = float("nan")
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    out = torch.full((5, 40), float("nan"), device=cuda_device)
    ops.router_topk_bwd(z, ids, gw, score, normalise, scale, grad_logits=out, dev_err=err)
    from moe_expert_epilogue_b200 import _abi
    assert int(err) == _abi.MOE_DEVERR_MAP
    known = torch.where(ids >= 40, torch.full_like(ids, -1), ids)
    want = _exact_grad(z, known, torch.nan_to_num(gw), score, normalise, scale)
    assert (out[2] == 0).all()
    assert ((out.double() - want).abs() <= 2e-5 * (1 + want.abs())).all()


@pytest.mark.parametrize("valid", [0, 3, 10, -2, 11])
def test_valid_tokens(cuda_device, valid):
    """Tokens at or past the device-resident count stay as they were; a count outside the
    tensor is clamped and reported."""
    z, g = _logits(10, 64, torch.bfloat16, 11, cuda_device)
    full_w, full_i = ops.router_topk_fwd(z, 8)
    gw = torch.randn(10, 8, generator=g, device=cuda_device)
    full_g = ops.router_topk_bwd(z, full_i, gw)
    n = torch.tensor([valid], dtype=torch.int32, device=cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    w = torch.full_like(full_w, 9.0)
    i = torch.full_like(full_i, 77)
    gl = torch.full_like(full_g, 9.0)
    ops.router_topk_fwd(z, 8, weights=w, ids=i, valid_tokens=n, dev_err=err)
    ops.router_topk_bwd(z, full_i, gw, grad_logits=gl, valid_tokens=n, dev_err=err)
    live = min(max(valid, 0), 10)
    assert torch.equal(w[:live], full_w[:live]) and (w[live:] == 9).all()
    assert torch.equal(i[:live], full_i[:live]) and (i[live:] == 77).all()
    assert torch.equal(gl[:live], full_g[:live]) and (gl[live:] == 9).all()
    from moe_expert_epilogue_b200 import _abi
    assert int(err) == (_abi.MOE_DEVERR_COUNT if valid in (-2, 11) else 0)


@pytest.mark.parametrize("dt", DTYPES)
def test_strides_and_alignment(cuda_device, dt):
    z, g = _logits(50, 64, dt, 13, cuda_device)
    gw = torch.randn(50, 8, generator=g, device=cuda_device)
    w, ids = ops.router_topk_fwd(z, 8)
    gl = ops.router_topk_bwd(z, ids, gw, normalise=False)
    for offset, pad in ((0, 8), (1, 0), (3, 5)):
        buf = torch.full((offset + 50 * (64 + pad),), 5.0, dtype=dt, device=cuda_device)
        zs = buf[offset:].view(50, 64 + pad)[:, :64]
        zs.copy_(z)
        w2, ids2 = ops.router_topk_fwd(zs, 8)
        assert torch.equal(w2, w) and torch.equal(ids2, ids)
        out = torch.full_like(buf, 4.0)
        gs = out[offset:].view(50, 64 + pad)[:, :64]
        ops.router_topk_bwd(zs, ids, gw, normalise=False, grad_logits=gs)
        assert torch.equal(gs, gl)
        assert (out[:offset] == 4).all() and (out[offset:].view(50, -1)[:, 64:] == 4).all()


def test_many_tokens_and_graph(cuda_device):
    z, g = _logits(20000, 64, torch.float32, 15, cuda_device)
    gw = torch.randn(20000, 8, generator=g, device=cuda_device)
    w, ids = ops.router_topk_fwd(z, 8)
    order = z.sort(dim=1, descending=True, stable=True).indices[:, :8].int()
    assert torch.equal(ids, order)
    gl = ops.router_topk_bwd(z, ids, gw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w2, i2 = ops.router_topk_fwd(z, 8)
        g2 = ops.router_topk_bwd(z, i2, gw)
    for t in (w2, i2, g2):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w2, w) and torch.equal(i2, ids) and torch.equal(g2, gl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w3, i3 = ops.router_topk_fwd(z, 8, stream=s)
    s.synchronize()
    assert torch.equal(w3, w) and torch.equal(i3, ids)


def test_weights_feed_the_activation_and_gradients_come_back(cuda_device):
    """The router's flat weights are the permuted activation's probs, and the router-weight
    multiply's grad_probs the router's grad_weights."""
    from moe_expert_epilogue_b200 import inputs
    t, k, e = 32, 4, 8
    z, g = _logits(t, e, torch.float32, 17, cuda_device)
    w, ids = ops.router_topk_fwd(z, k)
    rt = inputs.routing(t, k, e, 16, seed=1)
    x = inputs.permuted_activation_input(rt, 64, swiglu=True, seed=2).to(cuda_device)
    n = torch.tensor([rt.n_used], dtype=torch.int32, device=cuda_device)
    got = ops.act_with_probs_permuted(ops.MOE_ACT_SWIGLU, x, rt.permutation_map.to(cuda_device), n,
                                      w, zero_padding=True)
    pm = rt.permutation_map.to(cuda_device).long()
    p = torch.where(pm >= 0, w.view(-1)[pm.clamp(min=0)], torch.zeros((), device=cuda_device))
    gate, up = x.double().split(64, 1)
    want = torch.nn.functional.silu(gate) * up * p.double()[:, None]
    want = torch.where(pm[:, None] >= 0, want, torch.zeros_like(want))    # padding rows: zeros
    live = torch.arange(rt.max_rows, device=cuda_device) < rt.n_used
    # one bf16 rounding, and a sigmoid a few fp32 steps off: within a whole bf16 step
    assert ((got.double() - want).abs()[live] <= 2.0 ** -7 * want.abs()[live] + 1e-30).all()
    rows = torch.randn(t * k, 64, generator=g, device=cuda_device)
    go = torch.randn(t * k, 64, generator=g, device=cuda_device)
    _, gp = ops.router_weight_mul_bwd(go, rows, w.view(-1, 1))
    gl = ops.router_topk_bwd(z, ids, gp.view(t, k))
    want = _exact_grad(z, ids, (rows.double() * go.double()).sum(1).view(t, k), SOFT, True, 1.0)
    # grad_probs: 64 terms of order 1 summed in fp32, 1e-5 of a sum of order 50
    assert ((gl.double() - want).abs() <= 1e-4).all()


def _sorted_choice(z, k):
    """As _choose, for many tokens: a stable sort of the 64-bit values."""
    v, i = z.double().sort(dim=1, descending=True, stable=True)
    ids = torch.where(v[:, :k] == -INF, -1, i[:, :k]).int()
    return torch.cat([ids, ids.new_full((ids.shape[0], k - ids.shape[1]), -1)], 1)


@pytest.mark.parametrize("score,normalise,scale", MODES)
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("tokens,experts,top_k", [(4096, 8, 1), (4097, 64, 8), (5003, 161, 6),
                                                  (16390, 256, 8), (4100, 40, 5), (4099, 1024, 7),
                                                  (17001, 60, 3), (4098, 7, 7), (4101, 96, 9),
                                                  (8203, 161, 6), (8192, 8, 1), (8199, 1024, 8),
                                                  (8198, 7, 7)])
def test_many_tokens(cuda_device, tokens, experts, top_k, dt, score, normalise, scale):
    """Many tokens, some of them closed or with fewer open experts than choices; each has the
    bits that it has in a call of its own."""
    z, _ = _logits(tokens, experts, dt, tokens, cuda_device, masked=0.3)
    z[17] = -INF
    z[tokens - 1, 1:] = -INF
    w, ids = ops.router_topk_fwd(z, top_k, score, normalise, scale)
    assert torch.equal(ids, _sorted_choice(z, top_k))
    want = _weights(z, ids, score, normalise, scale)
    live = ids >= 0
    assert ((w.double() - want).abs() <= _tol(experts) * want.abs())[live].all()
    assert (w[~live] == 0).all()
    for a, b in ((0, 1), (16, 19), (40, 1040), (tokens - 70, tokens)):
        ws, js = ops.router_topk_fwd(z[a:b], top_k, score, normalise, scale)
        assert torch.equal(js, ids[a:b]) and torch.equal(ws, w[a:b])


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("experts", [56, 61, 256])
@pytest.mark.parametrize("tokens", [4500, 8500])
def test_many_tokens_strides_valid_and_nan(cuda_device, tokens, dt, experts):
    """Wider rows, rows off their alignment, NaN of either sign and zeros of either sign; tokens
    past the count keep what was there."""
    last = tokens - 3
    z, _ = _logits(tokens, experts, dt, 29, cuda_device)
    z[3, 5], z[4, 6], z[5, 2] = float("nan"), -float("nan"), INF
    z[6] = 0.0
    z[6, ::2] = -0.0
    valid = torch.tensor([last], dtype=torch.int32, device=cuda_device)
    w, ids = ops.router_topk_fwd(z, 8)
    assert ids[3, 0] == 5 and ids[4, 0] == 6 and ids[5, 0] == 2
    assert ids[6].tolist() == list(range(8))
    plain = torch.ones(tokens, dtype=torch.bool, device=cuda_device)
    plain[3:6] = False
    assert torch.equal(ids[plain], _sorted_choice(z[plain], 8))
    for wide, first in ((experts + 8, 0), (experts + 8, 8), (experts + 3, 1), (experts + 3, 3)):
        row = torch.full((tokens, wide), INF, dtype=dt, device=cuda_device)
        row[:, first:first + experts] = z
        w2 = torch.full_like(w, 7.0)
        i2 = torch.full_like(ids, 7)
        ops.router_topk_fwd(row[:, first:first + experts], 8, weights=w2, ids=i2,
                            valid_tokens=valid)
        assert torch.equal(i2[:last], ids[:last])
        assert torch.equal(w2[:last].view(torch.int32), w[:last].view(torch.int32))
        assert (w2[last:] == 7).all() and (i2[last:] == 7).all()


@pytest.mark.parametrize("score,normalise,scale", MODES)
@pytest.mark.parametrize("tokens,experts,top_k", [(1001, 64, 8), (333, 64, 9), (1003, 161, 6),
                                                  (77, 256, 17), (35, 512, 16), (21, 128, 8)])
def test_backward_bits_do_not_depend_on_the_batch(cuda_device, tokens, experts, top_k, score,
                                                  normalise, scale):
    z, g = _logits(tokens, experts, torch.float32, tokens, cuda_device, masked=0.2)
    ids = ops.router_topk_fwd(z, top_k)[1]
    gw = torch.randn(tokens, top_k, generator=g, device=cuda_device)
    whole = ops.router_topk_bwd(z, ids, gw, score, normalise, scale)
    for a, b in ((0, 1), (1, 4), (tokens - 5, tokens)):
        part = ops.router_topk_bwd(z[a:b], ids[a:b], gw[a:b], score, normalise, scale)
        assert torch.equal(part, whole[a:b])


@pytest.mark.parametrize("score,normalise,scale", MODES)
@pytest.mark.parametrize("tokens,experts,top_k", [(8199, 64, 8), (17000, 256, 8), (9000, 61, 3),
                                                  (8192, 1024, 8), (8192, 7, 7)])
def test_many_tokens_with_close_logits(cuda_device, tokens, experts, top_k, score, normalise,
                                       scale):
    """fp32 logits that differ in their last bits only, many of them equal, of either sign."""
    g = torch.Generator(device=cuda_device).manual_seed(tokens)
    z = 1.0 + torch.randint(0, 900, (tokens, experts), generator=g, device=cuda_device) * 2.0 ** -23
    z[::3] = -z[::3]
    z[1::5, ::2] = -INF
    z[7] = 0.0
    z[8, 1::2] = 0.5
    w, ids = ops.router_topk_fwd(z, top_k, score, normalise, scale)
    assert torch.equal(ids, _sorted_choice(z, top_k))
    want = _weights(z, ids, score, normalise, scale)
    live = ids >= 0
    assert ((w.double() - want).abs() <= _tol(experts) * want.abs())[live].all()
    ws, js = ops.router_topk_fwd(z[30:70], top_k, score, normalise, scale)
    assert torch.equal(js, ids[30:70]) and torch.equal(ws, w[30:70])


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("experts", [24, 65])
def test_many_tokens_of_extreme_values(cuda_device, dt, experts):
    """The type's lowest and largest values, subnormal ones and zeros, among closed experts."""
    info = torch.finfo(dt)
    least = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}[dt]
    values = torch.tensor([info.min, info.max, info.tiny, -info.tiny, least, -least, 3 * least, 0.0,
                           -0.0, -INF, INF], dtype=dt, device=cuda_device)
    g = torch.Generator(device=cuda_device).manual_seed(experts)
    z = values[torch.randint(0, values.numel(), (8200, experts), generator=g, device=cuda_device)]
    z[5] = info.min
    z[6] = -INF
    z[6, 3::7] = info.min
    ids = ops.router_topk_fwd(z, 8)[1]
    assert torch.equal(ids, _sorted_choice(z, 8))
    for a, b in ((0, 40), (8190, 8200)):
        assert torch.equal(ops.router_topk_fwd(z[a:b], 8)[1], ids[a:b])
    w = ops.router_topk_fwd(z, 8, SIG, False)[0]
    want = torch.sigmoid(z.double().gather(1, ids.long().clamp(min=0))) * (ids >= 0)
    assert ((w.double() - want).abs() <= 8 * U * want + 2.0 ** -126).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("experts", [40, 256, 1000])
def test_many_fp32_tokens_of_16_bit_values(cuda_device, dt, experts):
    """fp32 logits that came from a 16-bit type, with many equal ones: the same choice, and the
    same again with one logit's last bit set, which makes it the larger of its equals."""
    z, _ = _logits(8300, experts, dt, 51, cuda_device)
    z[5] = 1.0
    _, want = ops.router_topk_fwd(z, 8)
    z32 = z.float()
    w, ids = ops.router_topk_fwd(z32, 8)
    assert torch.equal(ids, want) and torch.equal(ids, _sorted_choice(z32, 8))
    bits = z32.view(torch.int32)
    up = torch.where(bits >= 0, bits | 1, bits)
    bits[:, experts - 3] = up[:, experts - 3]
    _, ids = ops.router_topk_fwd(z32, 8)
    assert torch.equal(ids, _sorted_choice(z32, 8)) and ids[5, 0] == experts - 3


@pytest.mark.parametrize("score,normalise,scale", MODES)
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("tokens,experts,top_k", [(16390, 40, 9), (20001, 161, 16),
                                                  (16385, 300, 12), (17001, 64, 17)])
def test_many_tokens_more_than_eight_choices(cuda_device, tokens, experts, top_k, dt, score,
                                             normalise, scale):
    """More than eight choices of more than 16384 tokens, two tokens side by side in a warp where
    their choices fit one; the last warp's second token is not there."""
    z, _ = _logits(tokens, experts, dt, tokens, cuda_device, masked=0.3)
    z[17] = -INF
    z[tokens - 1, 1:] = -INF
    w, ids = ops.router_topk_fwd(z, top_k, score, normalise, scale)
    assert torch.equal(ids, _sorted_choice(z, top_k))
    want = _weights(z, ids, score, normalise, scale)
    live = ids >= 0
    assert ((w.double() - want).abs() <= _tol(experts) * want.abs())[live].all()
    assert (w[~live] == 0).all()
    for a, b in ((0, 1), (16, 19), (tokens - 70, tokens)):
        ws, js = ops.router_topk_fwd(z[a:b], top_k, score, normalise, scale)
        assert torch.equal(js, ids[a:b]) and torch.equal(ws, w[a:b])
    valid = torch.tensor([tokens - 2], dtype=torch.int32, device=cuda_device)
    w2, i2 = torch.full_like(w, 7.0), torch.full_like(ids, 7)
    ops.router_topk_fwd(z, top_k, score, normalise, scale, weights=w2, ids=i2, valid_tokens=valid)
    assert torch.equal(i2[:-2], ids[:-2]) and torch.equal(w2[:-2], w[:-2])
    assert (w2[-2:] == 7).all() and (i2[-2:] == 7).all()
