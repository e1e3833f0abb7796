"""What a reading of the drafter's kernels has to show, on the source itself (no GPU here)."""
import os
import re

import pytest

import draft_token_verification_spec_b200 as sv
from draft_token_verification_spec_b200 import _build


def bodies(name):
    """The kernels of a file: (name, body), comments taken out."""
    with open(os.path.join(_build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    out = []
    for m in re.finditer(r"__global__[^{;]*?\b(\w+_kernel)\s*\(", text):
        a = text.index("{", m.end())
        depth, b = 0, a
        while True:
            depth += {"{": 1, "}": -1}.get(text[b], 0)
            if depth == 0:
                break
            b += 1
        out.append((m.group(1), text[a:b + 1]))
    return out


REMOTE = [(f, name, body) for f in ("distill.cuh", "sample.cuh", "row_stats.cuh")
          for name, body in bodies(f) if "map_shared_rank" in body]


@pytest.mark.parametrize("file,name,body", REMOTE, ids=[r[1] for r in REMOTE])
def test_remote_shared_memory_is_touched_only_once_its_block_runs(file, name, body):
    """A block of a cluster may read or write another's shared memory only after a barrier of the
    cluster that both have come to: all of them have started then."""
    before = body[:body.index("map_shared_rank")]
    arrive = [m.start() for m in re.finditer(r"cluster_arrive_started\(\)|cluster\(\)\.sync\(\)|\bcl\.sync\(\)", before)]
    wait = [m.start() for m in re.finditer(r"cluster_wait_started\(\)|cluster\(\)\.sync\(\)|\bcl\.sync\(\)", before)]
    assert arrive and wait and min(arrive) <= max(wait), name


def test_the_fused_row_kernel_is_among_them():
    assert "distill_row_kernel" in [r[1] for r in REMOTE]


@pytest.mark.parametrize("rows,V", [(65536, 1), (65536, 64), (65536, 1000), (4096, 2048)])
def test_workspaces_of_short_rows_hold_no_more_than_the_rows(rows, V):
    """A row of one tile: 16 bytes, eight warps' parts of 16, and a list of 8 bytes an entry, each of
    the three rounded up to 256 bytes for the call."""
    _build.build()
    most = rows * (16 + 8 * 16 + 8 * V) + 3 * 256
    assert 0 < sv.spec_sample_workspace_size(rows, V) <= most
    for k in {1, min(V, 50), min(V, 256)}:
        assert 0 < sv.spec_top_logits_workspace_size(rows, V, k) <= most
