"""Sizes that reach each kernel of the linear operator with 4-bit weights:
test_linear4_forms.py holds them against the plan, test_gpu_linear4_forms.py runs them."""

PAIRS = (("nv", "bf16"), ("nv", "fp16"), ("mx", "bf16"))

# {(form, rows of a in a tile / 16, its launch, gated): (M, N, K) of each of PAIRS}: tiles
# that are all whole, all cut along K, or some of each; written out in 16 bits
TILES = {
    ("tile", 1, "whole", False): ((17, 33, 416), (17, 33, 416), (17, 33, 416)),
    ("tile", 1, "cut", False): ((17, 33, 1056), (17, 33, 1056), (17, 33, 1440)),
    ("tile", 1, "both", False): ((5, 66001, 1440), (5, 66001, 1440), (5, 66001, 1440)),
    ("tile", 2, "whole", False): ((17, 33001, 416), (17, 33001, 416), (17, 33001, 416)),
    ("tile", 2, "cut", False): ((1021, 33, 4192), (1021, 33, 4192), (1021, 33, 4192)),
    ("tile", 2, "both", False): ((17, 66001, 1056), (17, 66001, 1056), (17, 66001, 1056)),
    ("tile", 4, "whole", False): ((33, 33001, 416), (33, 33001, 416), (33, 33001, 416)),
    ("tile", 4, "cut", False): ((33, 12001, 2112), (33, 12001, 4192), (803, 481, 4192)),
    ("tile", 4, "both", False): ((33, 66001, 800), (33, 66001, 1056), (33, 66001, 800)),
    ("tile", 8, "whole", False): ((97, 33001, 416), (97, 33001, 416), (97, 33001, 416)),
    ("tile", 8, "cut", False): ((65, 12001, 8224), (65, 12001, 8224), (97, 12001, 8224)),
    ("tile", 8, "both", False): ((65, 66001, 1440), (203, 66001, 672), (203, 66001, 800)),
    ("wide", 0, "", False): ((1021, 4223, 416), (1021, 4223, 416), (1021, 8193, 416)),
    ("tile", 1, "whole", True): ((17, 33, 416), (17, 33, 416), (17, 33, 416)),
    ("tile", 1, "cut", True): ((17, 33, 1056), (17, 33, 1056), (17, 33, 1440)),
    ("tile", 1, "both", True): ((5, 33001, 1440), (5, 33001, 1440), (5, 33001, 1440)),
    ("tile", 2, "whole", True): ((17, 16417, 416), (17, 16417, 416), (17, 16417, 416)),
    ("tile", 2, "cut", True): ((17, 6001, 1056), (451, 70, 4192), (451, 70, 4192)),
    ("tile", 2, "both", True): ((17, 33001, 1056), (17, 33001, 1056), (17, 33001, 1056)),
    ("tile", 4, "whole", True): ((33, 16417, 416), (33, 16417, 416), (33, 16417, 416)),
    ("tile", 4, "cut", True): ((33, 6001, 2112), (33, 6001, 4192), (33, 6001, 4192)),
    ("tile", 4, "both", True): ((33, 33001, 800), (33, 33001, 1056), (33, 33001, 800)),
    ("tile", 8, "whole", True): ((97, 16417, 416), (97, 16417, 416), (97, 16417, 416)),
    ("tile", 8, "cut", True): ((803, 481, 8224), (803, 481, 8224), (203, 2817, 8224)),
    ("tile", 8, "both", True): ((65, 66001, 672), (97, 66001, 672), (97, 66001, 800)),
    ("wide", 0, "", True): ((1021, 2111, 416), (1021, 2111, 416), (1021, 4223, 416)),
}

# few rows, and fp16 against UE8M0 scales in bands of 16, 32 and 64 rows and written out
OTHERS = tuple((form, dtype, "few", M, N, K, gated) for form, dtype in PAIRS for M in (1, 15) for N, K in ((70, 416), (705, 1440)) for gated in (False, True)) + \
    tuple(("mx", "fp16", "few" if M <= 64 else "wide", M, N, K, gated) for M in (5, 29, 61, 77, 301) for N, K in ((70, 416), (705, 1440))
          for gated in (False, True))


def all_cases():
    """(scales, a's type, form, 16-row fragments, launch, M, N, K, gated)"""
    for (form, fm, how, gated), sizes in TILES.items():
        for (scales, dtype), (M, N, K) in zip(PAIRS, sizes):
            yield scales, dtype, form, fm, how, M, N, K, gated
    for scales, dtype, form, M, N, K, gated in OTHERS:
        yield scales, dtype, form, 0, "", M, N, K, gated
