"""A wait inside the bf16 rows kernel that runs out (needs a GB300): one signal
after another between the kernel's warps is withheld on purpose.  The kernels
end by themselves, the call is reported, nothing but its outputs is written,
and the object runs a clean call with the same bits as before.  No GPU fault,
trap or hang is involved."""
import pytest
import torch

from test_gpu_cache import i32, sf  # noqa: F401
from test_gpu_cache_rows import rows_inputs, shared_inputs

pytestmark = pytest.mark.gpu

(PART, PART_READ, QUERIES, KEYS, KEYS_READ, VALUES, VALUES_READ, SCORES, WEIGHTS, LATE_WEIGHTS, TURN, OUTPUTS,
 MEET) = SIGNALS = range(1, 14)
PAD = 64   # rows of guard in front of and behind the outputs


def needed(rows, lens, G, nkv, hd):
    """The signals that some thread block waits for, by the split of sf_cache_index.h: a line of 24 units a tile and 5
    or 6 for each of its blocks, at least 6 units a thread block."""
    tiles, u = [], 0
    for r, n in zip(rows, lens):
        for x in list(range(0, r * G, 256)) * nkv if n else []:
            wide, nb = r * G - x > 128, -(-n // 128)
            tiles.append((u + 24, 6 if wide else 5, nb, wide))
            u += 24 + tiles[-1][1] * nb
    per = max(6, -(-u // torch.cuda.get_device_properties(0).multi_processor_count))
    blocks, parts, got = {}, {}, {PART, QUERIES, KEYS, VALUES, SCORES, WEIGHTS, LATE_WEIGHTS, OUTPUTS}
    for u0, cost, nb, wide in tiles:
        mine = {}
        for b in range(nb):
            c = (u0 + cost * b) // per
            mine[c] = mine.get(c, 0) + 1
        for c, m in mine.items():
            blocks[c], parts[c] = blocks.get(c, 0) + m, parts.get(c, 0) + 1
            got |= {TURN} if wide else {MEET} if m > 1 else set()
    if max(blocks.values()) > (2 if hd == 128 else 4):   # stages of the rings
        got |= {KEYS_READ, VALUES_READ}
    if max(parts.values()) >= 4:                         # parts handed out ahead, the end among them
        got |= {PART_READ}
    return got


def guarded(shape, dtype):
    return torch.full((shape[0] + 2 * PAD, *shape[1:]), 7.0, device="cuda", dtype=dtype)


def stalls(sf, a, call, signal, needed):
    """Run `call(out, lse)` cleanly, with the signal withheld, and cleanly again."""
    T = a["q"].shape[0]
    bufs = [guarded(a["q"].shape, torch.bfloat16), guarded(a["q"].shape[:2], torch.float32)]
    pools = a["k"].clone(), a["v"].clone()

    def run():
        for b in bufs:
            b.fill_(7.0)
        call(*[b[PAD:PAD + T] for b in bufs])
        torch.cuda.synchronize()
        for b in bufs:
            assert torch.all(b[:PAD] == 7.0) and torch.all(b[PAD + T:] == 7.0)
        assert torch.equal(a["k"].view(torch.int16), pools[0].view(torch.int16))
        assert torch.equal(a["v"].view(torch.int16), pools[1].view(torch.int16))
        return [b.clone() for b in bufs]

    good = run()
    a["c"].sync()
    sf.sf_cache_inject_stall(a["c"].cache, signal)
    got = run()
    if signal in needed:
        with pytest.raises(sf.SpecFoldError) as e:
            a["c"].sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and "wait" in str(e.value)
    else:
        a["c"].sync()
        assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])
    sf.sf_cache_inject_stall(a["c"].cache, 0)
    a["c"].sync()   # reported once
    for _ in range(2):
        again = run()
        a["c"].sync()
        assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
    a["c"].close()


ROWS = [
    # heads, page, rows, lens: wide tiles cut and whole, narrow ones, many parts of single blocks
    ((40, 8, 128), 32, [288] * 4, [4096] * 4),
    ((8, 8, 64), 16, [300, 7, 130], [3000, 2500, 2000]),
    ((16, 1, 128), 24, [8, 8], [30000, 20000]),
    ((32, 8, 128), 7, [20] * 100, [100] * 100),
]


@pytest.mark.parametrize("signal", SIGNALS)
@pytest.mark.parametrize("heads,page,rows,lens", ROWS)
def test_rows_end_when_a_wait_runs_out(sf, heads, page, rows, lens, signal):  # noqa: F811
    a = rows_inputs(sf, heads, "bf16", page, rows, lens, behind=0)
    table, n, st = i32(a["table"]), i32(a["lens"]), i32(a["starts"])
    stalls(sf, a, lambda out, lse: a["c"].attend_rows(a["q"], a["k"], a["v"], table, n, st, out=out, lse=lse), signal,
           needed(rows, lens, heads[0] // heads[1], heads[1], heads[2]))


@pytest.mark.parametrize("signal", SIGNALS)
@pytest.mark.parametrize("members,prefixes", [([9] * 4, [4096, 640, 5000, 1000]), ([70, 30], [9000, 300])])
def test_shared_ends_when_a_wait_runs_out(sf, members, prefixes, signal):  # noqa: F811
    a = shared_inputs(sf, (40, 8, 128), "bf16", 32, members, prefixes, 0, 0, [32] * sum(members))
    args = [i32(a[x]) for x in ("table", "lens", "ptable", "plens", "starts")]
    stalls(sf, a, lambda out, lse: a["c"].attend_shared(a["q"], a["k"], a["v"], *args, out=out, lse=lse), signal,
           needed(members, prefixes, 5, 8, 128))


def test_every_signal_is_needed_somewhere():
    assert set().union(*(needed(r, n, h[0] // h[1], h[1], h[2]) for h, _, r, n in ROWS)) == set(SIGNALS)


def test_stalls_refuse_other_signals(sf):  # noqa: F811
    a = rows_inputs(sf, (4, 2, 64), "bf16", 16, [1], [1])
    for signal in (-1, 14):
        with pytest.raises(sf.SpecFoldError) as e:
            sf.sf_cache_inject_stall(a["c"].cache, signal)
        assert e.value.status == sf.SF_ERR_INVALID_ARG
    with pytest.raises(sf.SpecFoldError):
        sf.sf_cache_inject_stall(None, 0)
    a["c"].close()
