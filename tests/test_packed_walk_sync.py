"""The packed attention's forward walks its work in shared memory: lane 0 of a warp steps, all
lanes read the step. Between the two stands a warp barrier on either side; shuffles order no
memory. The function is read from the source and its order of operations replayed for two
lanes, every read against every write of the other lane."""
import os
import re

SRC = os.path.join(os.path.dirname(__file__), "..", "video_diffusion_transformer_wan_b200", "csrc", "attn_packed_tc.cu")


def _events():
    """Barriers ("sync") and the step ("write") of one walk_next, in order; comments apart."""
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    body = re.search(r"bool walk_next\([^)]*\) \{(.*?)\n\}", text, re.S).group(1)
    return ["sync" if m == "__syncwarp()" else "write" for m in re.findall(r"__syncwarp\(\)|walk_step(?=\()", body)]


def test_a_step_is_ordered_with_the_reads_around_it():
    # lane 0 and another lane run: reads of piece n-1, walk_next, reads of piece n
    lane0, other = [], []
    for _ in range(3):
        for e in _events():
            lane0.append(e)
            if e == "sync":
                other.append(e)
        other.append("read")
    # the interval (number of barriers passed) of every access; two accesses of one interval race
    def intervals(trace, what):
        n, at = 0, []
        for e in trace:
            if e == "sync":
                n += 1
            elif e == what:
                at.append(n)
        return at

    writes, reads = intervals(lane0, "write"), intervals(other, "read")
    assert writes and reads
    assert not set(writes) & set(reads)
