"""CPU models of the wide and the e4m3 kernels' plans: every tile of a CTA-pair
product is done once and whole, rings of stages wait on the right phases, and the
few-row kernel's exchange puts each total where its reader looks, inside its
stages."""
import pytest

PAIRS, TILE = 76, 256


def ceil_div(a, b):
    return -(-a // b)


def pair_plan(rows, cols, tile_cols, nout, nchunk, may_split):
    mt, nt = ceil_div(rows, TILE), ceil_div(cols, tile_cols)
    tiles = mt * nt * nout
    plan = dict(mt=mt, nt=nt, nout=nout, whole=tiles, rest=0, splits=1, group=8, nchunk=nchunk)
    left = tiles % PAIRS
    if may_split and left:
        s = min(PAIRS // left, nchunk // 8, 16)
        if s > 1 and nchunk - nchunk // s >= 24:
            plan.update(whole=tiles - left, rest=left, splits=s)
    plan["ntiles"] = plan["whole"] + plan["rest"] * plan["splits"]
    return plan


def place(p, t):
    per = p["mt"] * p["nt"]
    o, t = divmod(t, per)
    g = t // (p["group"] * p["nt"])
    first = g * p["group"]
    gm = min(p["mt"] - first, p["group"])
    t -= first * p["nt"]
    return o, first + t % gm, t // gm


def tile_at(p, t):
    slot, c0, c1 = (-1 if t < p["whole"] else t - p["whole"]), 0, p["nchunk"]
    if slot >= 0:
        split = slot // p["rest"]
        t = p["whole"] + slot % p["rest"]
        c0, c1 = p["nchunk"] * split // p["splits"], p["nchunk"] * (split + 1) // p["splits"]
    return place(p, t), slot, c0, c1


@pytest.mark.parametrize("rows", [1, 256, 257, 333, 2100, 4096, 20000])
@pytest.mark.parametrize("cols,tile_cols,nout", [(1, 256, 1), (2560, 256, 1), (9728, 128, 1), (1000, 256, 2), (14336, 256, 2)])
@pytest.mark.parametrize("nchunk", [1, 8, 31, 76, 304])
def test_every_tile_once_and_whole(rows, cols, tile_cols, nout, nchunk):
    p = pair_plan(rows, cols, tile_cols, nout, nchunk, True)
    seen = {}
    for t in range(p["ntiles"]):
        at, slot, c0, c1 = tile_at(p, t)
        o, mi, ni = at
        assert o < nout and mi < p["mt"] and ni < p["nt"] and 0 <= c0 < c1 <= nchunk
        seen.setdefault(at, []).append((c0, c1, slot))
    assert len(seen) == p["mt"] * p["nt"] * nout
    slots = set()
    for parts in seen.values():
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == nchunk
        assert all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
        if len(parts) == 1:
            assert parts[0][2] == -1
        else:
            assert all(c1 - c0 >= 8 for c0, c1, _ in parts)
            slots.update(x[2] for x in parts)
    assert slots == set(range(p["rest"] * p["splits"])) and len(slots) <= PAIRS
    # the join finds the ranges of leftover tile i at slots i, i + rest, ..
    for i in range(p["rest"]):
        for s in range(p["splits"]):
            assert tile_at(p, p["whole"] + s * p["rest"] + i)[0] == place(p, p["whole"] + i)


@pytest.mark.parametrize("S", [3, 4, 6, 8])
@pytest.mark.parametrize("total", list(range(0, 30)))
@pytest.mark.parametrize("early", [False, True])
def test_ring_phases(S, total, early):
    """The producer's walk: a stage is filled again only after its products were read
    (barrier phase by phase), and the drain waits for the last fill of each stage.
    early: the first stages are filled before the loop."""
    done = [0] * S                                # completions of empty[] so far

    def passes(i, parity):                        # try_wait.parity: that phase has completed
        return (done[i] & 1) != parity

    pre = min(S, total) if early else 0
    fills = [0] * S
    for i in range(pre):
        fills[i] += 1
        done[i] += 1                              # read at once in this model
    st, phase, filled = (0, 0, pre) if pre == S else (pre, 1, pre)
    for _ in range(pre, total):
        assert passes(st, phase)
        if fills[st]:                             # not before its last fill was read
            done[st] -= 1
            assert not passes(st, phase)
            done[st] += 1
        fills[st] += 1
        done[st] += 1
        filled = min(S, filled + 1)
        st += 1
        if st == S:
            st, phase = 0, phase ^ 1
    for i in range(filled):
        at = st - (filled - i)
        parity = phase if at < 0 else phase ^ 1
        at %= S
        assert passes(at, parity)
        done[at] -= 1
        assert not passes(at, parity)
        done[at] += 1


@pytest.mark.parametrize("tn", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("mats", [1, 2])
def test_few_row_exchange(tn, mats):
    per_sm = 2 if tn <= 16 or (mats == 2 and tn <= 32) else 1
    stage = mats * 16384 + tn * 128
    scales = mats * tn * 4 * 4
    room = (113 if per_sm == 2 else 225) * 1024 - 1024 - 1024 - 2 * scales
    stages = min(8, room // stage)
    smem = 1024 + 1024 + 2 * scales + stages * stage
    assert stages >= 3 and smem <= 227 * 1024 and per_sm * (smem + 1024) <= 228 * 1024
    assert stage % 1024 == 0                       # every tile of a stage on the swizzle's 1024 bytes
    half_tokens = tn // 2
    for ks in range(1, 9):
        share = ceil_div(tn, ks)
        assert ks * mats * share * 128 * 4 <= stages * stage
        seen = {}
        for rank in range(ks):
            for half in (0, 1):
                owner, tok = divmod(half * half_tokens, share)
                for i in range(half_tokens):
                    for d in range(mats):
                        at = rank * mats * share + tok + d * share
                        assert owner < ks and at < ks * mats * share and (owner, at) not in seen
                        seen[owner, at] = (rank, d, half * half_tokens + i)
                    tok += 1
                    if tok == share:
                        owner, tok = owner + 1, 0
        for r in range(ks):                        # the reader's indexes
            for t in range(max(0, min(share, tn - r * share))):
                for s in range(ks):
                    for d in range(mats):
                        assert seen[r, (s * mats + d) * share + t] == (s, d, r * share + t)


CLUSTERS = [0, 152, 76, 46, 36, 28, 23, 15, 15]
TALL_COST = [(500, 210, 1, 50, 300, 350, 75, 1100), (1000, 290, 2, 57, 0, 2500, 276, 820)]
PAIR_COST = [(5300, 360, 130, 1800, 95), (6600, 330, 160, 0, 0)]


def tall_plan(M, N, K, dual):
    start, stage, stage_col, col, rnd, paired, rank, block = TALL_COST[dual]
    best = None
    for tn in (16, 32, 48) if dual else (16, 32, 48, 64, 80, 96, 112, 128):
        units, cols, chunks = ceil_div(N, 128) * ceil_div(M, tn), (1 + dual) * tn, ceil_div(K, 128)
        per_sm = 2 if tn <= 16 or (dual and tn <= 32) else 1
        for ks in range(1, min(8, chunks) + 1):
            ns = start + ceil_div(units, CLUSTERS[ks] * per_sm) * (
                ceil_div(chunks, ks) * (stage + stage_col * cols) + col * cols + rnd + (paired if per_sm == 2 else 0))
            ns += rank * ks + block * units * ks // 152
            if best is None or ns < best[0]:
                best = ns, tn, ks
        if tn >= M:
            break
    return best


def fp8_plan(M, N, K, dual):
    """("tall", tn, ks) or ("pair", plan)"""
    p = pair_plan(M, N, 128 if dual else 256, 1, ceil_div(K, 128), not dual)
    start, stage, full, join, join_slot = PAIR_COST[dual]
    stages = ceil_div(p["whole"], PAIRS) * p["nchunk"] + (ceil_div(p["nchunk"], p["splits"]) if p["rest"] else 0)
    ns = start + stages * (stage + full * min(p["ntiles"], PAIRS) // PAIRS)
    if p["rest"]:
        ns += join + join_slot * p["rest"] * p["splits"]
    tall = tall_plan(M, N, K, dual)
    return ("tall", *tall[1:]) if tall[0] < ns else ("pair", p)


def test_the_library_plans_as_the_model():
    """A product's workspace follows from its plan: none with the few-row kernel."""
    import memory_bound_glu_gb300 as mb
    seen = set()
    for M in (1, 16, 17, 64, 129, 333, 448, 500, 768, 1024, 2100, 4096):
        for N in (1, 300, 1000, 2000, 2560, 4096, 11008):
            for K in (128, 2048, 8192, 9728, 11008):
                kind, *rest = fp8_plan(M, N, K, 0)
                want = rest[0]["rest"] * rest[0]["splits"] * TILE * TILE * 4 if kind == "pair" else 0
                assert mb.matmul_fp8_workspace_bytes(M, N, K) == want, (M, N, K)
                seen.add((kind, want > 0))
    assert seen == {("tall", False), ("pair", False), ("pair", True)}


@pytest.mark.parametrize("dual", [0, 1])
def test_few_row_plans_are_launchable(dual):
    for M in (1, 8, 17, 100, 333, 1000, 5000, 100000):
        for N in (1, 128, 1000, 9728, 100000):
            for K in (1, 128, 129, 1000, 4096, 100000):
                ns, tn, ks = tall_plan(M, N, K, dual)
                assert ns > 0 and 1 <= ks <= min(8, ceil_div(K, 128)) and tn % 16 == 0 and tn <= 128
                c = ceil_div(K, 128)
                assert all(c * r // ks < c * (r + 1) // ks for r in range(ks))   # no block without a stage


def gemm_tokens(M, N, K):
    chunks, nt = ceil_div(K, 64), ceil_div(N, 128)
    tiles = nt * ceil_div(M, TILE)
    best, tn = 5760 + ceil_div(tiles, PAIRS) * chunks * (253 + 88 * min(tiles, PAIRS) // PAIRS), 0
    for t in range(32, TILE, 32):
        n = nt * ceil_div(M, t)
        ns = 4240 + ceil_div(n, PAIRS) * (chunks * (77 + 59 * min(n, PAIRS) // PAIRS) + chunks * t * 7 // 10 + t * 31 // 2)
        if ns < best:
            best, tn = ns, t
    return tn


def test_wide_forward_plan():
    """Narrow tiles for few rows and few tiles, 256-row tiles for long prompts."""
    assert {gemm_tokens(M, N, K) for M in (65, 100, 160, 200, 333, 400, 565, 700) for N in (300, 2500, 9728)
            for K in (264, 1000, 1528, 2560, 4096)} == {0, 32, 64, 96, 128, 160, 192, 224}
    for M in (1024, 2048, 2100, 4096, 8192):
        for N, K in ((9728, 2560), (14336, 4096), (4096, 2048), (11008, 4096)):
            assert gemm_tokens(M, N, K) == 0


@pytest.mark.parametrize("tn", range(32, 256, 32))
def test_wide_forward_exchange(tn):
    """A warp of g and its warp of u: each of the tile's values is used once, in the
    buffers' space, and every output has one writer."""
    seen = set()
    for half in (0, 1):
        for q in range(4):
            side, pairing = q >> 1, half * 2 + (q & 1)
            sets = 0
            for j in range(0, tn // 2, 16):
                mine = {pairing * 1024 + (sets & 1) * 512 + side * 256 + i * 32 + lane for i in range(8) for lane in (0, 31)}
                assert max(mine) < 8 * 32 * 17 and len(mine) == 16
                for i in range(8):
                    for lane in (0, 31):
                        at = (half * (tn // 2) + j + side * 8 + i, (q & 1) * 32 + lane)
                        assert at not in seen and at[0] < tn
                        seen.add(at)
                # what this warp hands over: the other side's eight
                assert (8 if side == 0 else 0) == (side ^ 1) * 8
                sets += 1
    assert len(seen) == tn * 4


def gemm_outputs(M, N, tn):
    tt = ceil_div(M, tn)
    places = ceil_div(ceil_div(N, 128) * tt, PAIRS) * PAIRS
    return next((wt for wt in (80, 96) if ceil_div(N, wt) * tt <= places), 128)


def test_wide_forward_outputs():
    """Every output in one lane of one tile, whatever the width; never more rounds."""
    assert {gemm_outputs(M, N, tn) for M in (17, 100, 333) for N in (300, 2504, 7000, 9728, 11008) for tn in (32, 128, 192)} == {80, 96, 128}
    for N in (1, 79, 80, 81, 300, 2504, 9728, 11008):
        for tn in (32, 192):
            wt = gemm_outputs(100, N, tn)
            assert ceil_div(ceil_div(N, wt) * ceil_div(100, tn), PAIRS) == ceil_div(ceil_div(N, 128) * ceil_div(100, tn), PAIRS)
            seen = [t * wt + rank * (wt // 2) + row for t in range(ceil_div(N, wt)) for rank in (0, 1) for row in range(64)
                    if row < wt // 2]
            assert sorted(n for n in seen if n < N) == list(range(N))
            assert wt // 2 % 8 == 0 and wt // 2 <= 64   # whole groups of the swizzle
