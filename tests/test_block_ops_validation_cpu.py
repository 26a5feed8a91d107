"""Argument checks of the layer norm and the router (not gpu): the C entry
points reject what they cannot run before anything is enqueued, the tensor
front end rejects mismatched tensors and never runs on the CPU."""
import pytest
import torch

from moe_expert_epilogue_b200 import _abi, build, ops

bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
FAKE = 0x10000  # never dereferenced
BF16, FP16, FP32 = _abi.MOE_BF16, _abi.MOE_FP16, _abi.MOE_FP32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _abi.lib()


def z(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


def _status(fn, *args):
    with pytest.raises(_abi.MoeError) as e:
        fn(*args)
    return e.value.status


def _device_error(fn):
    with pytest.raises(ValueError, match="CUDA device"):
        fn()


def test_layer_norm_fwd_status():
    f = _abi.moe_layer_norm_fwd

    def call(x=FAKE, w=FAKE, b=FAKE, y=FAKE, mean=FAKE, rstd=FAKE, rows=4, hidden=16, ld_x=16,
             ld_y=16, eps=1e-5, dt=BF16, w_dt=BF16):
        return _status(f, x, w, b, y, mean, rstd, rows, hidden, ld_x, ld_y, eps, dt, w_dt, 0)

    assert call(dt=9) == call(w_dt=FP16) == call(dt=FP32) == _abi.MOE_ERR_DTYPE
    assert call(rows=-1) == call(hidden=-1) == call(ld_x=15) == call(ld_y=15) == _abi.MOE_ERR_SHAPE
    assert call(rows=2 ** 40, ld_x=2 ** 40) == _abi.MOE_ERR_SHAPE
    for eps in (-1e-5, float("nan"), float("inf")):
        assert call(eps=eps) == _abi.MOE_ERR_LIMIT
    assert call(x=None) == call(w=None) == call(y=None) == _abi.MOE_ERR_NULL
    assert call(x=FAKE + 1) == call(y=FAKE + 1) == call(b=FAKE + 1) == _abi.MOE_ERR_ALIGN
    assert call(mean=FAKE + 2) == call(rstd=FAKE + 2) == call(w=FAKE + 2, w_dt=FP32) == \
        _abi.MOE_ERR_ALIGN
    f(None, None, None, None, None, None, 0, 16, 16, 16, 0.0, BF16, BF16, 0)   # no rows
    f(None, None, None, None, None, None, 4, 0, 0, 0, 0.0, BF16, FP32, 0)      # no columns


def test_layer_norm_bwd_status():
    size = _abi.moe_layer_norm_bwd_workspace
    assert size(0, 64) == 0 and size(1, 64) == 2 * 64 * 4
    assert size(10 ** 6, 64) == size(148, 64) == 148 * 2 * 64 * 4
    assert _status(size, -1, 4) == _status(size, 4, -1) == _abi.MOE_ERR_SHAPE

    def call(gy=FAKE, x=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, gx=FAKE, gw=FAKE, gb=FAKE, ws=FAKE,
             nbytes=2 * 4 * 16 * 4, rows=4, hidden=16, ld_gy=16, ld_x=16, ld_gx=16, dt=BF16,
             w_dt=FP32):
        return _status(_abi.moe_layer_norm_bwd, gy, x, w, mean, rstd, gx, gw, gb, ws, nbytes, rows,
                       hidden, ld_gy, ld_x, ld_gx, dt, w_dt, 0)

    assert call(w_dt=FP16) == _abi.MOE_ERR_DTYPE
    assert call(ld_gy=15) == call(ld_x=15) == call(ld_gx=15) == _abi.MOE_ERR_SHAPE
    assert call(nbytes=2 * 4 * 16 * 4 - 1) == _abi.MOE_ERR_SHAPE
    for k in ("gy", "x", "w", "mean", "rstd", "gx", "gw", "ws"):
        assert call(**{k: None}) == _abi.MOE_ERR_NULL
    for k in ("gy", "x", "w", "mean", "rstd", "gx", "gw", "gb", "ws"):
        assert call(**{k: FAKE + 1}) == _abi.MOE_ERR_ALIGN
    assert call(ws=FAKE + 8) == _abi.MOE_ERR_ALIGN
    assert call(rows=0, gw=None) == _abi.MOE_ERR_NULL        # the empty sums have a place to go


def test_router_status():
    def fwd(logits=FAKE, dt=FP32, w=FAKE, ids=FAKE, valid=FAKE, tokens=4, experts=64, top_k=8,
            ld=64, score=0, scale=1.0, err=None):
        return _status(_abi.moe_router_topk_fwd, logits, dt, w, ids, valid, tokens, experts, top_k,
                       ld, score, True, scale, err, 0)

    def bwd(logits=FAKE, dt=FP32, ids=FAKE, gw=FAKE, gl=FAKE, valid=FAKE, tokens=4, experts=64,
            top_k=8, ld=64, ld_g=64, score=0, scale=1.0, err=None):
        return _status(_abi.moe_router_topk_bwd, logits, dt, ids, gw, gl, valid, tokens, experts,
                       top_k, ld, ld_g, score, True, scale, err, 0)

    for call in (fwd, bwd):
        assert call(dt=5) == call(score=2) == _abi.MOE_ERR_DTYPE
        assert call(tokens=-1) == call(experts=0) == call(experts=1025, ld=1025) == \
            call(top_k=0) == call(top_k=33) == call(ld=63) == _abi.MOE_ERR_SHAPE
        assert call(experts=4, top_k=5) == _abi.MOE_ERR_SHAPE
        for scale in (float("nan"), float("inf")):
            assert call(scale=scale) == _abi.MOE_ERR_LIMIT
        assert call(logits=None) == call(ids=None) == _abi.MOE_ERR_NULL
        assert call(logits=FAKE + 2) == call(ids=FAKE + 2) == call(valid=FAKE + 2) == \
            call(err=FAKE + 2) == _abi.MOE_ERR_ALIGN
    assert fwd(w=None) == bwd(gw=None) == bwd(gl=None) == _abi.MOE_ERR_NULL
    assert bwd(ld_g=63) == _abi.MOE_ERR_SHAPE
    _abi.moe_router_topk_fwd(None, FP32, None, None, None, 0, 64, 8, 64, 0, True, 1.0, None, 0)
    _abi.moe_router_topk_bwd(None, FP32, None, None, None, None, 0, 64, 8, 64, 64, 0, True, 1.0,
                             None, 0)


def test_layer_norm_tensors():
    x, w = z(4, 16), z(16)
    with pytest.raises(ValueError, match="2-D"):
        ops.layer_norm_fwd(z(16), w)
    with pytest.raises(ValueError, match="elements"):
        ops.layer_norm_fwd(x, z(15))
    with pytest.raises(TypeError, match="dtype"):
        ops.layer_norm_fwd(x, z(16, dtype=torch.float16))
    with pytest.raises(TypeError, match="dtype"):
        ops.layer_norm_fwd(x, w, z(16, dtype=f32))              # bias as the weight
    with pytest.raises(TypeError, match="dtype"):
        ops.layer_norm_fwd(x.double(), w)
    with pytest.raises(ValueError, match="unit column stride"):
        ops.layer_norm_fwd(z(16, 4).t(), w)
    with pytest.raises(ValueError, match="non-overlapping"):
        ops.layer_norm_fwd(z(16).expand(4, 16), w)
    with pytest.raises(ValueError, match="shape"):
        ops.layer_norm_fwd(x, w, out=z(4, 15))
    with pytest.raises(ValueError, match="elements"):
        ops.layer_norm_fwd(x, w, mean=z(3, dtype=f32))
    _device_error(lambda: ops.layer_norm_fwd(x, w))
    m = z(4, dtype=f32)
    with pytest.raises(ValueError, match="shape"):
        ops.layer_norm_bwd(z(4, 15), x, w, m, m)
    with pytest.raises(TypeError, match="dtype"):
        ops.layer_norm_bwd(x, x, w, z(4), m)
    with pytest.raises(ValueError, match="elements"):
        ops.layer_norm_bwd(x, x, w, m, z(5, dtype=f32))
    with pytest.raises(TypeError, match="dtype"):
        ops.layer_norm_bwd(x, x, w, m, m, grad_weight=z(16, dtype=f32))
    with pytest.raises(TypeError, match="dtype"):
        ops.layer_norm_bwd(x, x, w, m, m, workspace=z(4096, dtype=f32))
    _device_error(lambda: ops.layer_norm_bwd(x, x, w, m, m))


def test_router_tensors():
    logits = z(4, 64, dtype=f32)
    with pytest.raises(ValueError, match="2-D"):
        ops.router_topk_fwd(z(64), 8)
    with pytest.raises(TypeError, match="dtype"):
        ops.router_topk_fwd(logits.double(), 8)
    with pytest.raises(ValueError, match="shape"):
        ops.router_topk_fwd(logits, 8, weights=z(4, 7, dtype=f32))
    with pytest.raises(TypeError, match="dtype"):
        ops.router_topk_fwd(logits, 8, ids=z(4, 8, dtype=torch.int64))
    with pytest.raises(TypeError, match="dtype"):
        ops.router_topk_fwd(logits, 8, valid_tokens=z(1, dtype=torch.int64))
    _device_error(lambda: ops.router_topk_fwd(logits, 8))
    ids, gw = z(4, 8, dtype=i32), z(4, 8, dtype=f32)
    with pytest.raises(ValueError, match="shape"):
        ops.router_topk_bwd(logits, ids[:3], gw)
    with pytest.raises(TypeError, match="dtype"):
        ops.router_topk_bwd(logits, ids, gw.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        ops.router_topk_bwd(logits, z(8, 4, dtype=i32).t(), gw)
    with pytest.raises(TypeError, match="dtype"):
        ops.router_topk_bwd(logits, ids, gw, grad_logits=z(4, 64))
    _device_error(lambda: ops.router_topk_bwd(logits, ids, gw))


def test_moe_layer_status():
    size = _abi.moe_layer_small_batch_workspace
    assert size(0, 64, 32, 4, 2) >= 256
    n = size(4, 64, 32, 8, 2)
    # logits, the two halves of the activation, the experts' rows
    assert n >= 256 + 4 * 8 * 4 + 4 * 2 * 2 * 32 * 2 + 4 * 2 * 64 * 4
    for bad in ((-1, 64, 32, 8, 2), (129, 64, 32, 8, 2), (128, 64, 32, 16, 9), (4, -1, 32, 8, 2),
                (4, 64, -1, 8, 2), (4, 64, 32, 0, 1), (4, 64, 32, 513, 2), (4, 64, 32, 8, 0),
                (4, 64, 32, 8, 9), (4, 64, 32, 40, 33), (4, 2 ** 20 + 1, 32, 8, 2)):
        assert _status(size, *bad) == _abi.MOE_ERR_SHAPE

    def call(x=FAKE, dt=BF16, rw=FAKE, rdt=BF16, logits=None, ldt=FP32, w1=FAKE, w2=FAKE,
             shared=FAKE, residual=FAKE, out=FAKE, tw=FAKE, ti=FAKE, valid=FAKE, ws=FAKE, nbytes=n,
             tokens=4, hidden=64, inter=32, experts=8, top_k=2, ld_x=64, ld_l=8, ld_s=64, ld_r=64,
             ld_o=64, score=0, scale=1.0, limit=7.0, err=None):
        return _status(_abi.moe_layer_small_batch, x, dt, rw, rdt, logits, ldt, w1, w2, shared,
                       residual, out, tw, ti, valid, ws, nbytes, tokens, hidden, inter, experts,
                       top_k, ld_x, ld_l, ld_s, ld_r, ld_o, score, True, scale, limit, err, 0)

    assert call(dt=FP32) == call(score=3) == call(rdt=FP16) == _abi.MOE_ERR_DTYPE
    assert call(rw=None, logits=FAKE, ldt=5) == _abi.MOE_ERR_DTYPE
    assert call(tokens=129) == call(experts=600) == call(top_k=9) == call(ld_x=63) == \
        call(ld_o=63) == call(ld_s=63) == call(ld_r=63) == call(nbytes=n - 1) == _abi.MOE_ERR_SHAPE
    assert call(rw=None, logits=FAKE, ld_l=7) == _abi.MOE_ERR_SHAPE
    assert call(limit=0.0) == call(limit=float("nan")) == call(scale=float("inf")) == \
        _abi.MOE_ERR_LIMIT
    for k in ("x", "rw", "w1", "w2", "out", "ws"):
        assert call(**{k: None}) == _abi.MOE_ERR_NULL
    assert call(logits=FAKE) == _abi.MOE_ERR_NULL          # both sources of the choice
    for k in ("x", "rw", "w1", "w2", "shared", "residual", "out", "tw", "ti", "valid", "ws", "err"):
        assert call(**{k: FAKE + 1}) == _abi.MOE_ERR_ALIGN
    assert call(ws=FAKE + 128) == call(rw=FAKE + 2, rdt=FP32) == _abi.MOE_ERR_ALIGN
    _abi.moe_layer_small_batch(None, BF16, None, BF16, None, FP32, None, None, None, None, None,
                               None, None, None, None, 0, 0, 64, 32, 8, 2, 64, 8, 0, 0, 64, 0,
                               True, 1.0, 7.0, None, 0)


def test_moe_layer_tensors():
    x, w1, w2, rw = z(4, 64), z(8, 64, 64), z(8, 64, 32), z(8, 64)
    f = ops.moe_layer_small_batch
    with pytest.raises(TypeError, match="dtype"):
        f(x.float(), w1, w2, 2, router_weight=rw)
    with pytest.raises(ValueError, match="3-D"):
        f(x, w1[0], w2, 2, router_weight=rw)
    with pytest.raises(ValueError, match="even"):
        f(x, w1[:, :63], w2, 2, router_weight=rw)
    with pytest.raises(ValueError, match="shape"):
        f(x, w1, w2[:, :, :31].contiguous(), 2, router_weight=rw)
    with pytest.raises(ValueError, match="contiguous"):
        f(x, w1, z(8, 32, 64).transpose(1, 2), 2, router_weight=rw)
    with pytest.raises(ValueError, match="either"):
        f(x, w1, w2, 2)
    with pytest.raises(ValueError, match="either"):
        f(x, w1, w2, 2, router_weight=rw, logits=z(4, 8))
    with pytest.raises(ValueError, match="shape"):
        f(x, w1, w2, 2, router_weight=z(7, 64))
    with pytest.raises(ValueError, match="shape"):
        f(x, w1, w2, 2, logits=z(4, 7, dtype=f32))
    with pytest.raises(TypeError, match="dtype"):
        f(x, w1, w2, 2, router_weight=rw, residual=z(4, 64, dtype=f32))
    with pytest.raises(ValueError, match="shape"):
        f(x, w1, w2, 2, router_weight=rw, topk_ids=z(4, 3, dtype=i32))
    with pytest.raises(ValueError, match="shape"):
        f(x, w1, w2, 2, router_weight=rw, out=z(4, 65))
    with pytest.raises(_abi.MoeError, match="SHAPE"):
        f(z(129, 64), w1, w2, 2, router_weight=rw)
    _device_error(lambda: f(x, w1, w2, 2, router_weight=rw))


def test_moe_layer_stalled_status():
    n = _abi.moe_layer_small_batch_workspace(4, 64, 32, 8, 2)

    def call(x=FAKE, logits=FAKE, w1=FAKE, w2=FAKE, out=FAKE, ws=FAKE, nbytes=n, tokens=4,
             hidden=64, inter=32, experts=8, top_k=2, stall=0, cycles=10 ** 5, err=FAKE):
        return _status(_abi.moe_test_layer_small_batch_stalled, x, logits, w1, w2, out, ws, nbytes,
                       tokens, hidden, inter, experts, top_k, stall, cycles, err, 0)

    for bad in (dict(stall=-1), dict(stall=6), dict(cycles=999), dict(cycles=2 ** 31 + 1),
                dict(nbytes=n - 1), dict(tokens=0), dict(tokens=129), dict(hidden=0),
                dict(inter=0), dict(experts=513), dict(top_k=9)):
        assert call(**bad) == _abi.MOE_ERR_SHAPE
    for k in ("x", "logits", "w1", "w2", "out", "ws", "err"):
        assert call(**{k: None}) == _abi.MOE_ERR_NULL
        assert call(**{k: FAKE + 1}) == _abi.MOE_ERR_ALIGN


def test_layer_norm_bwd_stalled_status():
    n = _abi.moe_layer_norm_bwd_workspace(40, 1024)

    def call(gy=FAKE, x=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, gx=FAKE, gw=FAKE, ws=FAKE, nbytes=n,
             rows=40, hidden=1024, stall=3, cycles=10 ** 5):
        return _status(_abi.moe_test_layer_norm_bwd_stalled, gy, x, w, mean, rstd, gx, gw, ws,
                       nbytes, rows, hidden, stall, cycles, 0)

    for bad in (dict(hidden=1020), dict(hidden=512), dict(hidden=2048), dict(hidden=8200),
                dict(rows=0), dict(stall=-1), dict(stall=40), dict(cycles=999),
                dict(cycles=2 ** 31 + 1), dict(nbytes=n - 1)):
        assert call(**bad) == _abi.MOE_ERR_SHAPE
    for k in ("gy", "x", "w", "mean", "rstd", "gx", "gw", "ws"):
        assert call(**{k: None}) == _abi.MOE_ERR_NULL
        assert call(**{k: FAKE + 1}) == _abi.MOE_ERR_ALIGN


def test_moe_layer_without_columns_status():
    n = _abi.moe_layer_small_batch_workspace(4, 0, 32, 8, 2)

    def call(rw=None, logits=FAKE, tw=FAKE, ti=FAKE, ws=FAKE, nbytes=n):
        return (_abi.moe_layer_small_batch, None, BF16, rw, BF16, logits, FP32, None, None, None,
                None, None, tw, ti, None, ws, nbytes, 4, 0, 32, 8, 2, 0, 8, 0, 0, 0, 0, True, 1.0,
                7.0, None, 0)

    assert _status(*call(ws=None)) == _status(*call(rw=FAKE)) == _abi.MOE_ERR_NULL
    assert _status(*call(nbytes=n - 1)) == _abi.MOE_ERR_SHAPE
    assert _status(*call(logits=FAKE + 2)) == _status(*call(ws=FAKE + 128)) == _abi.MOE_ERR_ALIGN
    f, *args = call(tw=None, ti=None, ws=None)                # no output at all
    f(*args)
