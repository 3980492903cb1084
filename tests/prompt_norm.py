"""How far outputs of the attention over whole prompts may be off in norm, a head at a time.  (The
bounds of prompt_ref.py hold every element in the worst case, with all roundings against it, and let
pass what is off by some percent everywhere; in norm roundings are independent.)

Each rounding to bf16 is spread over half a step, 2^-8 of a value at most, 2^-8 / sqrt(3) = 0.00226
in the mean square, and an output meets three at most: its own, that of P or dS, and out's in D.
Together 0.0039; 0.005 leaves a quarter for the fp32 sums and for heads of few elements."""
NORM = 0.005


def off(got, want):
    """||got - want|| / ||want|| over the last two axes."""
    err, size = (got.double() - want).norm(dim=(-2, -1)), want.norm(dim=(-2, -1))
    return (err / size.clamp(min=1e-300)).max().item()
