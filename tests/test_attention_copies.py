"""The end of the few-row attention's copies (no GPU needed): a CTA may not end under a copy into its shared memory, also where
a wait has given up.  Read from the source: the waits at the producer's end do not depend on what went well.  And their
arithmetic, restated: they cover every copy that was issued and may be on its way, and none that was not.
"""
import os
import random
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hadamard_rotation_gb300", "csrc")


def producer():
    with open(os.path.join(CSRC, "hq_kv_attend.cuh")) as f:
        source = f.read()
    text = source[source.index("if (warp == kWarps) {"):source.index("const int gq = lane >> 2")]
    return re.sub(r"//[^\n]*", "", text)


def test_waits_at_the_end_do_not_ask():
    text = producer()
    end = text[text.index("kv_cuts<D>(p.part)[blockIdx.x] = cut;"):]
    loop = end[end.index("for ("):end.rindex("}")]
    assert loop.count("mbar_wait(") == 1 and "if (" not in loop
    assert "for (uint32_t i = lane; i + last < kSlots && i < k; i += 32)" in loop
    given_up = text[text.index("if (!__all_sync(0xFFFFFFFFu, ok)) {"):]
    given_up = given_up[:given_up.index("}")]
    for part in ("if (issued) mbar_wait(smem_addr(&full[slot]), pass);",
                 "else if (lane < n && lane < kSlots && k + lane >= kSlots) mbar_wait(smem_addr(&full[slot]), pass ^ 1);", "last = n;", "break;"):
        assert part in given_up


def test_their_arithmetic():
    rng = random.Random(0)
    for _ in range(3000):
        slots, k, last, issued, now = rng.choice([21, 22, 55, 60, 90]), 0, 0, [], set()
        batches = [rng.randint(1, 32) for _ in range(rng.randint(1, 12))]
        fails = rng.random() < 0.7
        for b, n in enumerate(batches):
            lanes = range(n)
            if fails and b == len(batches) - 1:  # some lanes give up, all that would follow them in a place with them
                lanes = [lane for lane in lanes if lane < slots and rng.random() < 0.6]
                now = {k + lane for lane in lanes} | {k + lane - slots for lane in range(min(n, slots)) if lane not in lanes and k + lane >= slots}
                last = n
            issued += [k + lane for lane in lanes]
            if not last:
                k += n
        newest = {}  # a place is taken again only once its last copy has landed
        for seq in issued:
            newest[seq % slots] = seq
        covered = now | {k - 1 - i for i in range(slots) if i + last < slots and i < k}
        assert covered == set(newest.values())
