"""A kernel that gives up on a bounded wait leaves no copy in flight: what it issued is
drained, and its end waits for what cannot be asked about.  That path runs only when
something has gone wrong, so it is read from the sources."""
import os
import re

import pytest

import speculative_decoding_verify_kv_gb300 as va

CSRC = os.path.join(os.path.dirname(va.__file__), "csrc")


def body(name, code_only=True):
    with open(os.path.join(CSRC, f"va_latent_{name}.cu")) as f:
        text = f.read()
    if code_only:
        text = re.sub(r"//[^\n]*", "", text)
    start = text.index(f"latent_{name}_kernel(")
    return text[start:text.index("\n}\n", start)]


def block(text, at):
    """The braces that open behind `at`."""
    i = text.index("{", at)
    depth, j = 1, i + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
    return text[i:j]


def test_pair_drains_the_barriers_that_its_copies_land_on():
    text = body("pair")
    landing = {m.split("(")[0] if "VLAST" not in m else "PB_VLAST"
               for m in re.findall(r"expect_by\(one, (kfull\(|vfull\(|bar\(PB_VLAST)", text)}
    assert landing == {"kfull", "vfull", "PB_VLAST"}
    drains = [block(text, m.start()) for m in re.finditer(r"if \(\*abort_p && lane == 0\b", text)]
    assert len(drains) == 1
    assert all(name in drains[0] for name in landing)
    # A ragged last tile lands on each CTA's own barriers, so both wait for it.
    last, first = drains[0].index("PB_VLAST"), drains[0].index("rank == 0")
    assert last < first and "rank == 0" not in text[re.search(r"if \(\*abort_p && lane == 0", text).start():].split("{")[0]


def model(work, ragged, who, issued, units=4):
    """What the drain of a value warp asks for after `issued` of its units: (barrier, unit, parity)."""
    n = units // 2
    asked = []
    for k in range(max(0, issued - n), issued):
        i, u = k // n, who + 2 * (k % n)
        asked.append(("last", u, 0) if ragged and i == work - 1 else ("ring", u, i & 1))
    return asked


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("who", [0, 1])
def test_pair_value_drain_covers_what_was_issued(who, ragged):
    """The indices of the drain, restated, against a record of the copies: of each unit
    the last copy is asked for, on the barrier and in the phase that it was issued for."""
    text = re.sub(r"\s+", " ", body("pair"))
    for line in ("const int n = keys ? C::KU : C::VU / 2;", "const int i = k / n, u = keys ? k % n : who + 2 * (k % n);",
                 "issued = i * (C::VU / 2) + u / 2 + 1;", "for (int k = max(0, issued - n); k < issued; ++k)"):
        assert line in text
    for work in range(1, 6):
        record, count = {}, 0
        assert model(work, ragged, who, 0) == []
        for i in range(work):
            for u in range(who, 4, 2):
                alone = ragged and i == work - 1
                record[u] = ("last", u, 0) if alone else ("ring", u, i & 1)
                count += 1
                assert sorted(model(work, ragged, who, count)) == sorted(record.values())


def test_pair_gives_up_together():
    """Both CTAs of a pair learn of a failure before the closing barrier, and wait once
    more behind it."""
    text = body("pair")
    fail = block(text, text.index("auto fail"))
    assert "*abort_p = 1" in fail and re.search(r"store_at\(.*rank \^ 1, 1\)", fail)
    end = text[text.rindex("tc_fence_before();"):]
    assert re.search(r"cluster_sync_all\(\);\s*tc_fence_after\(\);\s*if \(\*abort_p\) \{\s*settle\(\);\s*cluster_sync_all\(\);\s*\}"
                     r"\s*if \(warp == 1\) tmem_dealloc_pair", end)


@pytest.mark.parametrize("name", ["rows", "umma", "prompt"])
def test_a_late_failure_is_waited_for(name):
    """A producer may issue its last copies and pass its own check just before another warp
    gives up: all warps look at the word behind the last barrier."""
    end = body(name)
    end = end[end.rindex("tc_fence_before();"):]
    assert re.search(r"__syncthreads\(\);\s*tc_fence_after\(\);\s*if \(\*abort_p\) settle\(\);\s*if \(warp == 1\) tmem_dealloc", end)
