"""Calls whose batch differs from what was planned for: more rows than the grid has row tiles in the kernel for many rows,
prompts beside single tokens in small batches, positions past the rotation tables.  Against the oracle."""
import numpy as np
import pytest

from oracle import kv8 as okv
from quantized_linear_layers_packed_amd import qlin
from tests.gpu_util import say, torch_cuda
from tests.test_gpu_kv8 import Setup, back, check_attention, check_round16, run_append, run_attention, to16

pytestmark = pytest.mark.gpu

F16, BF16 = qlin.QLIN_F16, qlin.QLIN_BF16


@pytest.mark.parametrize("max_kv", [1, 700, 6000])
@pytest.mark.parametrize("dtype,D,P,Hk,G,max_new,new,kv,window,sinks", [
    (F16, 64, 16, 2, 4, 20, [300, 3, 41], [700, 90, 600], 0, 0),          # 1200 rows, one row tile of 128 in the grid
    (BF16, 128, 64, 1, 8, 10, [150, 1], [1900, 300], 0, 0),               # 1200 rows, 256 to a tile
    (F16, 256, 32, 1, 2, 35, [301], [640], 0, 0),                         # 602 rows, 128 to a tile
    (BF16, 64, 128, 1, 8, 33, [200, 90], [1500, 1111], 300, 70),          # three row tiles of the grid are walked on from
    (F16, 128, 32, 1, 8, 9, [90, 1, 0, 9, 2, 40, 1, 5, 130], [300, 2500, 9, 9, 2, 1900, 63, 5, 700], 0, 0),
])
def test_rows_past_the_planned_tiles_of_the_kernel_for_many_rows(dtype, D, P, Hk, G, max_new, new, kv, window, sinks, max_kv):
    """max_new plans for that kernel, and for fewer of its row tiles than the longest sequence has; long planned lengths
    split the first ones, whose partial results the later ones must leave alone."""
    say(f"kv8 attention past the plan: D={D} G={G} max_new={max_new} of {new}, max_kv={max_kv} of {kv}")
    s = Setup(41, D, P, Hk, new, kv, max_new=max_new, max_kv=max_kv)
    Q = s.rng.standard_normal((s.T, Hk * G, D))
    first = back(check_attention(s, G, dtype, Q=Q, window=window, sinks=sinks))
    assert np.array_equal(back(run_attention(s, G, dtype, Q=Q, window=window, sinks=sinks)[0]), first)


@pytest.mark.parametrize("dtype,D,G", [(F16, 128, 8), (BF16, 64, 4), (F16, 256, 2)])
@pytest.mark.parametrize("new,kv", [([90, 1], [300, 3000]), ([1, 200, 1, 1], [1500, 200, 7, 2100]), ([1, 5, 1, 130, 1, 40, 2], [900, 64, 2, 1000, 77, 40, 3000])])
def test_prompts_beside_single_tokens_in_small_batches(dtype, D, G, new, kv):
    check_attention(Setup(42, D, 32, 1, new, kv), G, dtype)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("new,kv", [([1, 1], [41, 100]), ([30, 70], [60, 90])])
def test_positions_past_the_rotation_tables_use_their_last_row(pairs, new, kv):
    torch = torch_cuda()
    say(f"kv8 append past the tables: new={new} kv={kv} pairs={pairs}")
    s = Setup(43, 64, 16, 2, new, kv)
    d, x = to16(s.rng.standard_normal((s.T, 8, 64)), BF16)
    cos, sin = okv.rope_tables(40, 32)
    out = torch.full((s.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    qlin.qlin_kv8_append(s.cache, s.batch, d[:, :4], d[:, 4:6], d[:, 6:], BF16, 4, torch.from_numpy(cos).cuda(),
                         torch.from_numpy(sin).cuda(), 32, qlin.QLIN_ROPE_PAIRS if pairs else qlin.QLIN_ROPE_HALF, out)
    ref = okv.append(s.k, s.v, s.scales, s.offsets, s.kv_lens, s.table, x[:, :4], x[:, 4:6], x[:, 6:], cos, sin, 32, pairs)
    s.check_cache()
    check_round16(out, ref, BF16)


@pytest.mark.parametrize("max_new", [1, 33])
def test_appends_past_the_planned_pages(max_new):
    """More pages and more query tokens than the grid was made for, one sequence's after another's."""
    for D, P in ((64, 16), (256, 128)):
        say(f"kv8 append past the plan: D={D} P={P} max_new={max_new}")
        s = Setup(44, D, P, 2, [500, 1, 129], [700, 20, 129], max_new=max_new, max_kv=1)
        q, q_ref = run_append(s, 6, F16, D, False)
        s.check_cache()
        check_round16(q, q_ref, F16)
        torch = torch_cuda()
        K, V = (torch.full((s.T, 2, D), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
        qlin.qlin_kv8_gather(s.cache, s.batch, K, V, F16)
        refs = [np.concatenate([okv.values(s.k, s.v, s.scales, s.table[b], m, h)[i][m - n:] for b, (n, m) in enumerate(zip(s.new, s.kv))])
                for i in (0, 1) for h in (0, 1)]
        for got, ref in ((K, refs[:2]), (V, refs[2:])):                     # fp64, which holds scale * code, rounded once
            assert np.array_equal(back(got), np.stack(ref, 1).astype(np.float16))
