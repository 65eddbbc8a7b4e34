"""GPU test of the placement that the workgroup renumbering (xcd_remap) rests on, whichever XCD a
launch's first workgroup goes to: workgroups are dealt out to the eight XCDs in turn, and with the
renumbering each XCD's tasks are one contiguous range."""
import numpy as np
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2048, 1920, 128 * 13])
def test_each_xcd_runs_one_range_of_tasks(n):
    import block_swizzle_tile_amd as bst
    base = dict(tile=(128, 128), offset=2, direction="zn")
    tasks = (n // 128) ** 2
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            maps = [bst.tile_map(1, n, n, bst.make_sched(xcd_remap=r, grid=tasks, **base)).cpu().numpy()
                    for r in (0, 1)]
        for got, remap in zip(maps, (0, 1)):
            wg, xcc = got[:, 7], got[:, 6]
            say("first workgroup's XCD", int(xcc[np.argmin(wg)]), "tasks", tasks, "remap", remap)
            assert sorted(wg.tolist()) == list(range(tasks))
            # in turn, from wherever the launch begins
            assert np.unique((xcc - wg) % 8).size == 1
        # one range of tasks an XCD: the XCD changes seven times along the task order, to each once
        xcc = maps[1][:, 6]
        starts = np.concatenate([[0], np.flatnonzero(np.diff(xcc)) + 1])
        assert starts.size == 8 and np.unique(xcc[starts]).size == 8
        assert np.ptp(np.bincount(xcc, minlength=8)) <= 1
