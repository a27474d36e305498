"""Launches of the largest sizes that calls accept: fewer than 2^32 threads each, and together they cover the call. Without
a GPU, from the launches that the library asks the runtime for."""
import pytest

import launch_shim

LIMIT = 1 << 32  # threads of one launch, a limit of the runtime's own
ROWS, Q, SCALE = 1 << 40, 1 << 42, 1 << 44
UNSUPPORTED = "3"


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    return launch_shim.build(str(tmp_path_factory.mktemp("shim")))


@pytest.mark.parametrize("n,parts,width", [
    (1, 1, 8), (1000, 2, 264), (2 ** 29 - 32, 1, 8), (2 ** 29 - 31, 1, 8), (2 ** 29, 1, 8), (2 ** 30 - 1, 1, 8),
    ((2 ** 30 - 1) // 3, 3, 8), ((2 ** 30 - 1) // 9, 3, 264), (1, 2, 2 ** 31 - 128), (1, 2, 2 ** 31 - 120),
    (20, 3, 2 ** 31 - 8)])
def test_codes_of_many_groups(shim, n, parts, width):
    code = f"""
for dtype in (0, 1):
    say(lib.lrmoe_checkpoint(i64({n}), {parts}, {width}, dtype, vp({ROWS}), vp({Q}), vp({SCALE}), None))
    say(lib.lrmoe_restore(i64({n}), {parts}, {width}, vp({Q}), vp({SCALE}), dtype, vp({ROWS}), None))
"""
    groups = (width + 127) // 128
    calls = launch_shim.run(shim, code)
    assert len(calls) == 4
    for i, (status, launches) in enumerate(calls):
        size, saves = (4, 2)[i // 2], i % 2 == 0
        assert status == "0" and launches
        done = 0  # rows of one part
        for at in launches:
            assert at.threads < LIMIT and at.grid[1:] == [1, 1]
            rows, q, scale = at.args[1:] if saves else (at.args[3], *at.args[1:3])
            assert (rows - ROWS, q - Q, scale - SCALE) == (done * width * size, done * width, done * groups * 2)
            units = at.args[0] & 0xFFFFFFFF  # Place begins with them
            assert units % groups == 0 and at.threads // 8 - 32 < units <= at.threads // 8
            done += units // groups
        assert done == n * parts


PROBLEM = """
class Problem(ctypes.Structure):
    _fields_ = [(n, i32) for n in ("E", "T", "K", "D", "F", "swiglu", "dtype", "reserved")] + [
        ("N", i64), ("seg_off", vp), ("quota", vp)]


def problem(T, K, D, F, N, swiglu=1, dtype=0, kept=None):
    kept = N if kept is None else kept
    p = Problem(E=1, T=T, K=K, D=D, F=F, N=N, swiglu=swiglu, dtype=dtype)
    p.keep = (i64 * 2)(0, N), (i32 * 1)(kept)
    p.seg_off, p.quota = (ctypes.cast(a, vp) for a in p.keep)
    return ctypes.byref(p)


def score(p, ws=1 << 60):
    return lib.lrmoe_score_checkpoint(p, vp(4096), vp(4096), vp(4096), vp(4096), vp(4096), vp(4096), vp(4096),
                                      ctypes.c_size_t(ws), None)


def compact(p):
    return lib.lrmoe_compact_checkpoint(p, vp(4096), vp(4096), vp(4096), vp(4096), vp(4096), None)
"""


@pytest.mark.parametrize("dtype,D", [(0, 64), (1, 64), (0, 2 ** 29), (1, 2 ** 30), (0, 2 ** 31 - 8), (1, 2 ** 31 - 8)])
def test_words_of_a_wide_row(shim, dtype, D):
    """A row's words of 16 bytes, counted without its bytes passing 32 bits."""
    code = PROBLEM + f"""
p = problem(40000, 1, {D}, {D}, 40000, swiglu=0, dtype={dtype})
say(score(p))
say(score(p, ws=8 * 40064))
say(lib.lrmoe_score(p, *[vp(4096)] * 6, ctypes.c_size_t(1 << 30), None))
say(lib.lrmoe_compact_weighted(p, *[vp(4096)] * 4, None))
"""
    words = D // (8 if dtype else 4)
    calls = launch_shim.run(shim, code)
    assert [status for status, _ in calls] == ["0"] * 4
    (_, fused), (_, two), (_, plain), (_, compact) = calls
    low = lambda launch, i: launch.args[i] & 0xFFFFFFFF  # noqa: E731
    if 40000 * words > 2 ** 21:
        assert low(fused[0], 3) == words and low(two[0], 2) == words
    assert low(plain[0], 2) == low(compact[0], 2) == words


@pytest.mark.parametrize("T,K,N,D,ws,ok", [
    (2 ** 26 - 8, 8, 2 ** 28 - 16, 64, 1 << 60, True), (2 ** 26 - 8, 8, 2 ** 28 - 15, 64, 1 << 60, False),
    (2 ** 26 - 8, 8, 2 ** 28, 64, 8 << 26, False), (2 ** 24, 32, 2 ** 29 - 32, 8, 1 << 60, False),
    (2 ** 26 - 4, 1, 2 ** 22, 64, 8 << 26, True), (2 ** 26 - 4, 1, 2 ** 22, 64, 1 << 60, True),
    (2 ** 26 - 3, 1, 2 ** 22, 64, 8 << 28, False), (2 ** 27, 1, 2 ** 22, 64, 1 << 60, False),
    (2 ** 30, 1, 1000, 64, 8 << 30, True)])  # few pairs read their tokens' rows themselves
def test_scores_of_many_pairs(shim, T, K, N, D, ws, ok):
    for dtype in (0, 1):
        code = PROBLEM + f"say(score(problem({T}, {K}, {D}, 8, {N}, dtype={dtype}), ws={ws}))"
        (status, launches), = launch_shim.run(shim, code)
        if ok:
            assert status == "0" and launches and all(at.threads < LIMIT for at in launches)
        else:
            assert status == UNSUPPORTED and not launches


@pytest.mark.parametrize("kept,ok", [(1, True), (2 ** 28 - 16, True), (2 ** 28 - 15, False), (2 ** 28, False),
                                     (2 ** 31 - 32, False)])
def test_many_retained_pairs(shim, kept, ok):
    code = PROBLEM + f"say(compact(problem({2 ** 26 - 1}, 32, 8, 8, {2 ** 31 - 32}, kept={kept})))"
    (status, launches), = launch_shim.run(shim, code)
    if ok:
        assert status == "0" and len(launches) == 1 and launches[0].threads < LIMIT and launches[0].args[0] == kept
    else:
        assert status == UNSUPPORTED and not launches


ROUTER = """
class Router(ctypes.Structure):
    _fields_ = [(n, i32) for n in ("T", "E", "K", "first", "local", "dtype", "renorm", "reserved")] + [("scale", f32)]


class Scoring(ctypes.Structure):
    _fields_ = [(n, i32) for n in ("score", "groups", "top_groups", "group_best")]


note(0)
F, ws = vp(4096), ctypes.c_size_t(1 << 60)
"""


@pytest.mark.parametrize("T", [2 ** 26 - 4, 2 ** 26 - 3, 2 ** 26 - 1])
@pytest.mark.parametrize("E,K", [(1024, 8), (513, 31), (512, 8), (64, 20), (8, 4), (1, 1)])
def test_router_of_most_tokens(shim, T, E, K):
    code = PROBLEM + ROUTER + f"""
r = ctypes.byref(Router(T={T}, E={E}, K={K}, local={E}, dtype=1, renorm=1, scale=1.0))
for score in (0, 1):
    c = ctypes.byref(Scoring(score, 1, 1, 1))
    say(f"route {{lib.lrmoe_route_scored(r, c, F, F, None, F, F, F, F, F, F, F, F, F, ws, None)}}")
    for n in (1, min(2 ** 21 - 1, (2 ** 31 - 1) // {E})):
        say(f"loss {{lib.lrmoe_balance_loss_scored(r, c, F, None, F, F, n, f32(1), F, F, F, F, F, ws, None)}}")
    say(f"gradient {{lib.lrmoe_route_bwd_scored(r, c, F, None, F, F, F, i64(5), F, 3, F, F, None, F, None)}}")
say(f"weights {{lib.lrmoe_alpha_grad(problem({T}, {K}, 8, 8, 1000), F, F, F, F, None, F, None)}}")
"""
    for text, launches in launch_shim.run(shim, code):
        call, status = text.split()
        if T > 2 ** 26 - 4 and (call == "weights" or call == "gradient" and E > 512):
            assert status == UNSUPPORTED and not launches, text
        else:
            assert status == "0" and launches and all(at.threads < LIMIT for at in launches), text


@pytest.mark.parametrize("T,E,launches", [
    (128, 1024, 1), (129, 8, 2), (3073, 1024, 2), (4096, 1024, 2), (4096, 777, 2), (4097, 1024, 3), (32768, 128, 2),
    (65536, 128, 3), (24000, 256, 2), (32768, 256, 3), (40000, 96, 3), (700_000, 64, 2), (4_000_000, 8, 2), (6_000_000, 8, 3)])
def test_launches_of_routing(shim, T, E, launches):
    """Top-K alone, with the placing, or with a scan of the counts between: as each was measured to be faster."""
    code = ROUTER + f"""
r = ctypes.byref(Router(T={T}, E={E}, K=1, local={E}, dtype=0, renorm=1, scale=1.0))
say(lib.lrmoe_route(r, F, None, F, F, F, F, F, F, F, F, F, ws, None))
"""
    (status, found), = launch_shim.run(shim, code)
    assert status == "0" and len(found) == launches
