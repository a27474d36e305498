"""The router's operators and AdamW without a GPU: refusals (host checks before any launch), and
the fp64 definitions against differences and counts of their own."""
import ctypes

import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from load_recalibrated_expert_amd import _lib
from oracle import router_oracle as ro

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1008)


def _router(**kw):
    d = dict(T=10, E=16, K=4, first=0, local=16, dtype=_lib.F32, renorm=0, reserved=0, scale=1.0)
    d.update(kw)
    return _lib.CRouter(**d)


def _size(r, n_seq=1):
    n = ctypes.c_size_t(0)
    return _lib.load().lrmoe_router_workspace_size(ctypes.byref(r), n_seq, ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,expect", [
    ({}, _lib.OK), (dict(T=0), _lib.OK), (dict(E=1024, local=1024, K=32), _lib.OK), (dict(first=15, local=1), _lib.OK),
    (dict(T=-1), _lib.ERR_INVALID_ARG), (dict(E=0), _lib.ERR_INVALID_ARG), (dict(K=0), _lib.ERR_INVALID_ARG),
    (dict(K=17), _lib.ERR_INVALID_ARG), (dict(first=-1), _lib.ERR_INVALID_ARG), (dict(local=0), _lib.ERR_INVALID_ARG),
    (dict(first=1, local=16), _lib.ERR_INVALID_ARG), (dict(first=2 ** 31 - 1, local=1), _lib.ERR_INVALID_ARG),
    (dict(renorm=2), _lib.ERR_INVALID_ARG), (dict(reserved=1), _lib.ERR_INVALID_ARG),
    (dict(scale=float("nan")), _lib.ERR_INVALID_ARG), (dict(scale=float("inf")), _lib.ERR_INVALID_ARG),
    (dict(dtype=2), _lib.ERR_UNSUPPORTED), (dict(E=1025, local=1025), _lib.ERR_UNSUPPORTED),
    (dict(E=64, K=33, local=64), _lib.ERR_UNSUPPORTED), (dict(T=2 ** 30, K=2), _lib.ERR_UNSUPPORTED),
])
def test_router_checks(kw, expect):
    st, n = _size(_router(**kw))
    assert st == expect and (n >= 256 if st == _lib.OK else n == 0)


def test_sequence_counts_are_checked():
    assert _size(_router(), 0)[0] == _lib.ERR_INVALID_ARG
    assert _size(_router(), 2 ** 30)[0] == _lib.ERR_UNSUPPORTED
    assert _size(_router(), 1000)[1] > _size(_router(), 1)[1]


def test_sizes_past_one_launch_are_refused():
    """A launch takes fewer than 2^32 threads along a dimension: T < 2^26 tokens, n_seq < 2^21."""
    lib, few = _lib.load(), dict(E=2, K=1, local=2)
    assert _size(_router(T=2 ** 26 - 1, **few))[0] == _lib.OK
    assert _size(_router(T=2 ** 26, **few))[0] == _lib.ERR_UNSUPPORTED
    assert _size(_router(**few), 2 ** 21 - 1)[0] == _lib.OK
    assert _size(_router(**few), 2 ** 21)[0] == _lib.ERR_UNSUPPORTED
    r = _router(**few)
    assert lib.lrmoe_balance_loss(ctypes.byref(r), FAKE, None, FAKE, FAKE, 2 ** 21, 0.1, *([FAKE] * 5), 2 ** 40,
                                  None) == _lib.ERR_UNSUPPORTED
    assert lib.lrmoe_route_bwd(ctypes.byref(r), FAKE, None, FAKE, None, None, 0, FAKE, 2 ** 21, FAKE, FAKE, None, FAKE,
                               None) == _lib.ERR_UNSUPPORTED
    p, keep = _lib.make_problem_struct(2, 2 ** 26, 2, 8, 8, True, _lib.BF16, [0, 5, 9], [5, 4])
    assert lib.lrmoe_alpha_grad(ctypes.byref(p), *([FAKE] * 4), None, FAKE, None) == _lib.ERR_UNSUPPORTED


def test_route_refusals():
    lib, r = _lib.load(), _router()
    n = _size(r)[1]

    def call(ptrs=None, ws=FAKE, nb=n, router=r, mask=None):
        p = dict(logits=FAKE, idx=FAKE, w=FAKE, counts=FAKE, seg_off=FAKE, tok=FAKE, slot=FAKE, alpha=FAKE, pmap=FAKE)
        p.update(ptrs or {})
        return lib.lrmoe_route(ctypes.byref(router), p["logits"], mask, p["idx"], p["w"], p["counts"], p["seg_off"],
                               p["tok"], p["slot"], p["alpha"], p["pmap"], ws, nb, None)

    for name in ("logits", "idx", "w", "counts", "seg_off", "tok", "slot", "alpha", "pmap"):
        assert call({name: None}) == _lib.ERR_INVALID_ARG, name
    assert call({"logits": ODD}) == _lib.ERR_INVALID_ARG
    assert call(ws=None) == _lib.ERR_WORKSPACE
    assert call(nb=0) == _lib.ERR_WORKSPACE
    assert call(router=_router(K=0)) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_route(None, *([FAKE] * 11), n, None) == _lib.ERR_INVALID_ARG


def test_balance_refusals():
    lib, r = _lib.load(), _router()
    n = _size(r, 3)[1]

    def call(logits=FAKE, idx=FAKE, off=FAKE, n_seq=3, coef=0.1, counts=FAKE, psum=FAKE, norm=FAKE, loss=FAKE, ws=FAKE,
             nb=n):
        return lib.lrmoe_balance_loss(ctypes.byref(r), logits, None, idx, off, n_seq, coef, counts, psum, norm, loss,
                                      ws, nb, None)

    for kw in (dict(logits=None), dict(logits=ODD), dict(idx=None), dict(off=None), dict(n_seq=0), dict(n_seq=-1),
               dict(coef=float("nan")), dict(counts=None), dict(psum=None), dict(norm=None), dict(loss=None)):
        assert call(**kw) == _lib.ERR_INVALID_ARG, kw
    assert call(ws=None) == _lib.ERR_WORKSPACE
    assert call(nb=16) == _lib.ERR_WORKSPACE


def test_route_bwd_refusals():
    lib, r = _lib.load(), _router()

    def call(logits=FAKE, idx=FAKE, dalpha=FAKE, pmap=FAKE, n_pairs=5, off=FAKE, n_seq=2, counts=FAKE, norm=FAKE,
             out=FAKE):
        return lib.lrmoe_route_bwd(ctypes.byref(r), logits, None, idx, dalpha, pmap, n_pairs, off, n_seq, counts, norm,
                                   None, out, None)

    for kw in (dict(logits=None), dict(logits=ODD), dict(out=None), dict(out=ODD), dict(idx=None), dict(n_pairs=-1),
               dict(counts=None), dict(off=None), dict(n_seq=0)):
        assert call(**kw) == _lib.ERR_INVALID_ARG, kw


def test_alpha_grad_refusals():
    lib = _lib.load()
    p, keep = _lib.make_problem_struct(2, 6, 2, 64, 32, True, _lib.BF16, [0, 5, 9], [5, 4])
    q, keep2 = _lib.make_problem_struct(2, 6, 2, 60, 32, True, _lib.BF16, [0, 5, 9], [5, 4])
    for i in range(4):
        a = [FAKE] * 4
        a[i] = None
        assert lib.lrmoe_alpha_grad(ctypes.byref(p), *a, None, FAKE, None) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_alpha_grad(ctypes.byref(p), *([FAKE] * 4), None, None, None) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_alpha_grad(ctypes.byref(p), ODD, FAKE, FAKE, FAKE, None, FAKE, None) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_alpha_grad(ctypes.byref(q), *([FAKE] * 4), None, FAKE, None) == _lib.ERR_UNSUPPORTED


def _config(**kw):
    d = dict(w_dtype=_lib.BF16, grad_dtype=_lib.F32, master=1, state_bits=8, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
             weight_decay=0.1, grad_scale=1.0, step=1, seed=3, reserved=0)
    d.update(kw)
    return _lib.CAdamwConfig(**d)


@pytest.mark.parametrize("kw,expect", [
    ({}, _lib.OK), (dict(master=0, w_dtype=_lib.F32, state_bits=32), _lib.OK), (dict(beta1=0.0), _lib.OK),
    (dict(w_dtype=_lib.F32), _lib.ERR_UNSUPPORTED), (dict(w_dtype=3), _lib.ERR_UNSUPPORTED),
    (dict(grad_dtype=2), _lib.ERR_UNSUPPORTED), (dict(state_bits=16), _lib.ERR_UNSUPPORTED),
    (dict(master=2), _lib.ERR_INVALID_ARG), (dict(lr=float("nan")), _lib.ERR_INVALID_ARG),
    (dict(beta1=1.0), _lib.ERR_INVALID_ARG), (dict(beta2=-0.1), _lib.ERR_INVALID_ARG),
    (dict(beta2=float("nan")), _lib.ERR_INVALID_ARG), (dict(eps=-1.0), _lib.ERR_INVALID_ARG),
    (dict(weight_decay=float("inf")), _lib.ERR_INVALID_ARG), (dict(grad_scale=float("inf")), _lib.ERR_INVALID_ARG),
    (dict(step=0), _lib.ERR_INVALID_ARG), (dict(reserved=1), _lib.ERR_INVALID_ARG),
])
def test_adamw_config_checks(kw, expect):
    lib, s = _lib.load(), _lib.CAdamwScalars()
    assert lib.lrmoe_adamw_step_scalars(ctypes.byref(_config(**kw)), ctypes.byref(s)) == expect
    assert lib.lrmoe_adamw(None, 0, ctypes.byref(_config(**kw)), None, None, None) == expect  # no tensors: nothing to launch


def test_adamw_scalars():
    lib, s = _lib.load(), _lib.CAdamwScalars()
    assert lib.lrmoe_adamw_step_scalars(None, ctypes.byref(s)) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_adamw_step_scalars(ctypes.byref(_config(step=7)), None) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_adamw_step_scalars(ctypes.byref(_config(step=7, grad_scale=0.5)), ctypes.byref(s)) == _lib.OK
    f = np.float32
    assert (s.decay, s.lr, s.grad_scale) == (f(1 - 1e-3 * 0.1), f(1e-3), 0.5)
    assert s.c1 == f(1 / (1 - 0.9 ** 7)) and abs(s.c2 - 1 / np.sqrt(1 - 0.999 ** 7)) <= 2 ** -23 * s.c2
    assert s.key == int(ro.mix((3 + int(ro.mix(7))) & 0xFFFFFFFF))


def test_adamw_tensor_refusals():
    lib = _lib.load()
    good = dict(w=0x1000, master=0x2000, grad=0x3000, m=0x4000, v=0x5000, m_scale=0x6000, v_scale=0x7000, n=300, first=0)

    def call(cfg=None, **kw):
        t = (_lib.CAdamwTensor * 2)(_lib.CAdamwTensor(n=0), _lib.CAdamwTensor(**{**good, **kw}))
        return lib.lrmoe_adamw(t, 2, ctypes.byref(cfg or _config()), None, None, None)

    for kw in (dict(w=None), dict(master=None), dict(grad=None), dict(m=None), dict(v=None), dict(m_scale=None),
               dict(v_scale=None), dict(n=-1), dict(first=-256), dict(first=100), dict(w=0x1008), dict(master=0x2004),
               dict(grad=0x3002), dict(m=0x4002), dict(v_scale=0x7001)):
        assert call(**kw) == _lib.ERR_INVALID_ARG, kw
    assert call(n=2 ** 37) == _lib.ERR_UNSUPPORTED
    c32 = _config(state_bits=32)
    assert call(c32) == _lib.ERR_INVALID_ARG  # scales given to 32-bit states
    assert call(c32, m_scale=None, v_scale=None, m=0x4004) == _lib.ERR_INVALID_ARG  # 32-bit states: 16 bytes
    assert lib.lrmoe_adamw(None, 1, ctypes.byref(_config()), None, None, None) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_adamw(None, -1, ctypes.byref(_config()), None, None, None) == _lib.ERR_INVALID_ARG


def test_adamw_plan():
    """The plan's size, its refusals, and its contents: the tensors that have elements and their first
    chunks of a whole number of elements each."""
    lib = _lib.load()
    c = _config(state_bits=32)
    sizes = [5, 0, 100000, 4096, 1]
    t = (_lib.CAdamwTensor * 5)(*[_lib.CAdamwTensor(w=0x1000 * (i + 1), master=0x90000, grad=0x90000, m=0x90000, v=0x90000,
                                                   n=n) for i, n in enumerate(sizes)])
    n = ctypes.c_size_t(0)
    assert lib.lrmoe_adamw_plan(t, 5, ctypes.byref(c), None, None) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_adamw_plan(t, 5, None, None, ctypes.byref(n)) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_adamw_plan(None, 5, ctypes.byref(c), None, ctypes.byref(n)) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_adamw_plan(t, 5, ctypes.byref(c), None, ctypes.byref(n)) == _lib.OK
    need = n.value
    buf = (ctypes.c_uint8 * need)()
    n.value = need - 1
    assert lib.lrmoe_adamw_plan(t, 5, ctypes.byref(c), buf, ctypes.byref(n)) == _lib.ERR_WORKSPACE
    n.value = need
    assert lib.lrmoe_adamw_plan(t, 5, ctypes.byref(c), buf, ctypes.byref(n)) == _lib.OK and n.value == need
    size = ctypes.sizeof(_lib.CAdamwTensor)
    live = (_lib.CAdamwTensor * 4).from_buffer(buf)
    assert [e.n for e in live] == [5, 100000, 4096, 1] and [e.w for e in live] == [0x1000, 0x3000, 0x4000, 0x5000]
    first = np.frombuffer(buf, np.uint32, 4, 4 * size).tolist()
    assert first[0] == 0 and first[1] == 1  # five elements are one chunk
    chunk = 4096 // (first[3] - first[2])
    assert first[2] == 1 + -(-100000 // chunk)
    assert lib.lrmoe_adamw(t, 5, ctypes.byref(c), ctypes.c_void_p(0x1008), None, None) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_adamw(t, 5, ctypes.byref(c), None, ctypes.c_void_p(0x1002), None) == _lib.ERR_INVALID_ARG


def test_python_refusals():
    for kw in (dict(T=4, E=4, K=5), dict(T=4, E=4, K=2, first=4), dict(T=4, E=4, K=2, first=1, local=4)):
        with pytest.raises(lr.LrmoeError):
            lr.Router(device="cpu", **kw)
    w = [torch.zeros(300), torch.zeros(40)]
    g = [torch.zeros(300), torch.zeros(40)]
    lr.AdamW(w, grads=g)
    lr.AdamW(w, grads=g, bits=8)
    for kw in (dict(bits=4), dict(weights=[]), dict(weights=[w[0], w[1].bfloat16()]), dict(weights=[w[0].half()]),
               dict(grads=[g[0]]), dict(grads=[g[0], g[1][:7]]), dict(masters=[w[0]]), dict(m=[w[0], w[1][:4]]),
               dict(weights=[w[0], w[0]]), dict(weights=[w[0], w[0][128:168]]), dict(bits=8, first=[0]),
               dict(bits=8, m=[torch.zeros(300), torch.zeros(40)])):
        with pytest.raises(ValueError):
            lr.AdamW(**{**dict(weights=w, grads=g), **kw})
    for kw in (dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(lr=float("nan"))):
        with pytest.raises(lr.LrmoeError):
            lr.AdamW(w, grads=g, **kw)
    with pytest.raises(lr.LrmoeError):  # f32 weights are their own masters
        lr.AdamW(w, masters=[torch.zeros(300), torch.zeros(40)])
    with pytest.raises(ValueError):
        lr.AdamW(w).step()
    with pytest.raises(ValueError):
        lr.AdamW(w, grads=g).step_captured()


def test_a_refused_advance_counts_no_step():
    opt = lr.AdamW([torch.zeros(40)], grads=[torch.zeros(40)], step=6)
    for bad in (float("nan"), float("inf"), None):
        with pytest.raises((lr.LrmoeError, TypeError)):
            opt.advance(grad_scale=bad)
        assert opt.t == 6
    opt.lr = float("nan")
    with pytest.raises(lr.LrmoeError):
        opt.advance()
    assert opt.t == 6
    opt.lr = 1e-3
    opt.advance()
    assert opt.t == 7


# ----------------------------------------------------------------------- the definitions themselves

def _logits(rng, T, E):
    return rng.standard_normal((T, E)) * 2


@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(renorm):
    rng = np.random.default_rng(3)
    T, E, K = 7, 9, 3
    x = _logits(rng, T, E)
    y = rng.standard_normal((T, K))
    f = ro.route(x, K, renorm=renorm, scale=1.7)
    dx, _ = ro.route_bwd(x, f["idx"], y=y, renorm=renorm, scale=1.7)
    h = 1e-6
    for t, e in [(0, 0), (3, 5), (6, 8)] + [(2, int(f["idx"][2, k])) for k in range(K)]:
        d = []
        for s in (h, -h):
            z = x.copy()
            z[t, e] += s
            g = ro.route(z, K, renorm=renorm, scale=1.7)
            assert np.array_equal(g["idx"], f["idx"])
            d.append((g["w"] * y).sum())
        assert abs((d[0] - d[1]) / (2 * h) - dx[t, e]) < 1e-7


def test_balance_gradient_against_differences():
    rng = np.random.default_rng(4)
    T, E, K = 23, 6, 2
    x, mask, off = _logits(rng, T, E), (rng.random(T) < 0.8).astype(np.uint8), [0, 5, 5, 17, 23]
    idx = ro.route(x, K, mask=mask)["idx"]
    b = ro.balance(x, idx, 0.3, mask=mask, seq_off=off)
    dx, _ = ro.route_bwd(x, idx, counts=b["counts"], norm=b["norm"], gloss=0.9, mask=mask, seq_off=off)
    h = 1e-6
    for t in range(T):
        e = int(rng.integers(E))
        d = []
        for s in (h, -h):
            z = x.copy()
            z[t, e] += s
            d.append(0.9 * ro.balance(z, idx, 0.3, mask=mask, seq_off=off)["loss"])
        assert abs((d[0] - d[1]) / (2 * h) - dx[t, e]) < 1e-7


def test_balance_loss_is_coef_for_a_uniform_router():
    """Equal probabilities: E sum_e f_e P_e = 1 whatever the choices."""
    T, E, K = 40, 8, 2
    idx = np.stack([np.arange(T) % E, (np.arange(T) + 3) % E], 1).astype(np.int32)
    assert abs(ro.balance(np.zeros((T, E)), idx, 0.01, seq_off=[0, 11, 40])["loss"] - 0.01) < 1e-15


def test_rounding_is_unbiased_and_bounded():
    rng = np.random.default_rng(5)
    n, rounds = 512, 400
    x = (rng.standard_normal(n) * np.exp2(rng.integers(-12, 1, n))).astype(np.float32)
    got = []
    for t in range(rounds):
        lo, hi = ro.random_bits(n, 256 * 7, 11, t + 1)
        q, s = ro.quantise(x, lo, True)
        v = ro.dequantise(q, s)
        step = np.maximum(np.exp2(np.floor(np.log2(np.abs(x) / np.repeat(s, 256))) - 3), 2.0 ** -9) * np.repeat(s, 256)
        assert np.all(np.abs(v - x) <= step * (1 + 1e-6))
        codes = torch.from_numpy(q).to(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(codes, q)  # e4m3 holds every value
        got.append((v - x) / step)
    mean = np.mean(got, 0)  # each term is in [-1, 1] with a deviation of at most 1/2
    assert np.all(np.abs(mean) < 6 * 0.5 / np.sqrt(rounds)), np.abs(mean).max()
    assert abs(np.mean(mean)) < 6 * 0.5 / np.sqrt(rounds * n)


def test_root_never_rounds_to_zero():
    x = np.concatenate([np.full(1, 1.0), np.full(200, 1e-7), np.zeros(55)]).astype(np.float32)
    for t in range(5):
        q, s = ro.quantise(x, ro.random_bits(256, 0, 1, t)[1], False)
        assert np.all((q > 0) == (x > 0))


def test_counter_has_64_bits():
    a, b = ro.random_bits(600, 2 ** 32 - 256, 5, 9), ro.random_bits(344, 2 ** 32, 5, 9)
    assert np.array_equal(a[0][256:], b[0]) and not np.array_equal(a[0][256:], ro.random_bits(344, 0, 5, 9)[0])


def test_gradients_that_overlap_what_adamw_writes_are_refused():
    """A gradient inside the weights, the masters or the states would be read while it is overwritten."""
    flat, g = torch.zeros(1000), [torch.zeros(300), torch.zeros(40)]
    w = [flat[:300], flat[400:440]]
    for grads in (w, [g[0], w[1]], [flat[100:400], g[1]], [g[0], flat[401:441]], [g[0], flat[361:401]]):
        with pytest.raises(ValueError):
            lr.AdamW(w, grads=grads)
    m = torch.zeros(300)
    with pytest.raises(ValueError):
        lr.AdamW([w[0]], grads=[m], m=[m])
    half = [t.bfloat16() for t in w]
    opt = lr.AdamW(half, masters=w, grads=g)
    with pytest.raises(ValueError):
        opt.bind(w)
    assert opt.grads == g
    lr.AdamW(w, grads=[flat[440:740], flat[300:340]])  # beside them
    lr.AdamW([w[0], torch.zeros(300)], grads=[g[0], g[0]])  # one gradient for two weights is only read
    lr.AdamW([flat[:0], w[1]], grads=[flat[400:400], g[1]])  # without elements nothing overlaps


@pytest.mark.parametrize("E,dtype,off,ok", [
    (17, _lib.F32, 4, True), (17, _lib.F32, 2, False), (18, _lib.F32, 8, True), (18, _lib.F32, 4, False),
    (20, _lib.F32, 16, True), (20, _lib.F32, 8, False), (17, _lib.BF16, 2, True), (17, _lib.BF16, 1, False),
    (20, _lib.BF16, 8, True), (20, _lib.BF16, 4, False), (1, _lib.BF16, 2, True), (1024, _lib.F32, 8, False)])
def test_logits_may_start_at_any_row(E, dtype, off, ok):
    """A view that starts at a later row of an aligned buffer is as aligned as a row is long. What is taken
    goes on to the workspace's check."""
    lib, r = _lib.load(), _router(E=E, local=E, K=1, dtype=dtype)
    at = ctypes.c_void_p(0x1000 + off)
    want = _lib.ERR_WORKSPACE if ok else _lib.ERR_INVALID_ARG
    assert lib.lrmoe_route(ctypes.byref(r), at, None, *([FAKE] * 8), None, 0, None) == want
    assert lib.lrmoe_balance_loss(ctypes.byref(r), at, None, FAKE, None, 1, 0.1, *([FAKE] * 4), None, 0, None) == want
    if not ok:
        for pair in ((at, FAKE), (FAKE, at)):
            assert lib.lrmoe_route_bwd(ctypes.byref(r), pair[0], None, FAKE, FAKE, None, 0, None, 1, None, None, None,
                                       pair[1], None) == want


@pytest.mark.parametrize("kw", [dict(lr=1e39), dict(lr=-1e39), dict(weight_decay=1e300, lr=1e300), dict(eps=1e39),
                                dict(grad_scale=1e39), dict(lr=1e20, weight_decay=1e20)])
def test_adamw_values_that_f32_does_not_hold_are_refused(kw):
    """The kernel takes them in f32, where they would be infinite and end every weight."""
    lib, s = _lib.load(), _lib.CAdamwScalars()
    c = _config(**kw)
    assert lib.lrmoe_adamw_step_scalars(ctypes.byref(c), ctypes.byref(s)) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_adamw(None, 0, ctypes.byref(c), None, None, None) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_adamw_plan(None, 0, ctypes.byref(c), None, ctypes.byref(ctypes.c_size_t(0))) == _lib.ERR_INVALID_ARG
