"""The attention kernels' source, on the CPU: instructions of whole warps stand behind a warp sync.

PTX leaves a `.sync.aligned` instruction undefined for a warp that is not converged (tensor-memory loads, stores and their
waits, allocation, register shares).  Loops, branches and stores that go by lane may leave a warp split, so every such
instruction has to follow a __syncwarp(), with no condition between them but those on values that a warp shares."""
import os
import re

SRC = os.path.join(os.path.dirname(__file__), "..", "speculative_decoding_verification_09_gb300", "csrc",
                   "attention.cuh")
# what a condition between a sync and an instruction of a whole warp may name: a tile's width, counters of
# loops with constant bounds, template arguments, and the layout's constants
SHARED = {"int", "x", "i", "w", "SYNC", "PAIR", "NQ", "DP", "constexpr"}
UNSYNCED = re.compile(r"\btm_\w+<false>\s*\(|\bhalf_done\(\)")  # (half_done begins with an unsynced wait)


def statements(text):
    """The source without comments, cut behind every ; { and } outside strings."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    out, at = [], 0
    for m in re.finditer(r'"(?:\\.|[^"\\])*"|[;{}]', text):
        if m.group() in ";{}":
            out.append(" ".join(text[at:m.end()].split()))
            at = m.end()
    return out


def raw(text):
    """(number, faults) of asm statements with an instruction of a whole warp that do not directly follow a sync, one
    that a template argument may leave out, or another such instruction."""
    bad, n, safe = [], 0, False
    for s in statements(text):
        whole_warp = ".sync.aligned" in s
        if whole_warp:
            n += 1
            # (an asm statement by itself: a condition before it would be a branch between the two)
            if not safe or not s.startswith("asm volatile("):
                bad.append(s[:120])
        safe = whole_warp or s in ("__syncwarp();", "if (SYNC) __syncwarp();")
    return n, bad


def names(s):
    return set(re.findall(r"[A-Za-z_]\w*", s))


def by_lane(s):
    """Whether a statement branches, or may, on something outside SHARED."""
    conditions = re.findall(r"\b(?:if|for|while)\b(?: constexpr)? \(((?:[^()]|\([^()]*\))*)", s)
    return any(not names(c) <= SHARED for c in conditions) or "?" in s or "&&" in s or "||" in s


def unsynced(text):
    """(number, faults) of calls without a sync of their own between which and the last sync a condition may split the
    warp."""
    text, bad, n = statements(text), [], 0
    for k, s in enumerate(text):
        if not UNSYNCED.search(s):
            continue
        n += 1
        j = k
        while j >= 0:
            if by_lane(text[j]):
                bad.append((s[:80], text[j][:80]))
                break
            if j < k and (text[j] == "__syncwarp();" or
                          (re.search(r"\btm_(ld|st|wait)\w*\(", text[j]) and "void" not in text[j])):
                break
            j -= 1
        else:
            bad.append((s[:80], "no sync"))
    return n, bad


def test_whole_warp_instructions_follow_a_warp_sync():
    n, bad = raw(open(SRC).read())
    assert n >= 10 and not bad, bad


def test_calls_without_their_own_sync_follow_one():
    text = open(SRC).read()
    text = text[text.index("sv_attn(const __grid_constant__"):]
    n, bad = unsynced(text)
    assert n >= 8 and not bad, bad
    # and what stands between them by name does not branch by lane
    for name in ("chunk = [&](int x)", "half_done = [&]"):
        body = text[text.index(name):]
        body = statements(body[:body.index("\n            };" if "chunk" in name else "\n        };")])
        assert len(body) > 3 and not any(by_lane(s) for s in body), (name, body)


def test_the_rules_find_a_missing_sync():
    ok = 'void f() { __syncwarp(); asm volatile("x.sync.aligned;" ::: "memory"); asm volatile("y.sync.aligned;"); }'
    assert raw(ok) == (2, [])
    assert len(raw(ok.replace("__syncwarp();", ""))[1]) == 1
    assert len(raw(ok.replace("__syncwarp();", "__syncwarp(); if (lane == 0) { g(); }"))[1]) == 1
    assert len(raw(ok.replace("__syncwarp();", "__syncwarp(); if (lane)"))[1]) == 1
    assert raw(ok.replace("__syncwarp();", "// __syncwarp();\n"))[1]
    ok = "{ __syncwarp(); for (int x = 0; x < 4; ++x) if (x * 32 < w) tm_ld32<false>(ts, r); tm_wait_ld<false>(r); }"
    assert unsynced(ok) == (2, [])
    assert unsynced(ok.replace("__syncwarp();", ""))[1]
    assert unsynced(ok.replace("w)", "row)"))[1]
    assert unsynced(ok.replace("tm_wait", "if (lane == 0) mbar_arrive(b); tm_wait"))[1]
    assert unsynced(ok.replace("tm_wait", "a = b ? 1 : 2; tm_wait"))[1]
